"""Paged key/value cache cases for the tests: device tensors, their host copies and the error bounds."""
import numpy as np
import torch

from oracle import kv as okv

PAGE = 64
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0, torch.float8_e4m3fn: 2.0 ** -10}


def host(t):
    return t.double().cpu().numpy()


def axis_of(rot, n_axes):
    return [i % n_axes for i in range(rot // 2)]


def inv_freq(rot):
    return (10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)).float().cuda()


class Case:
    """A cache with `old` tokens a sequence and `new` ones to come; pools hold NaN where no token is."""

    def __init__(self, csa, old, new, H, kv_heads, dim, dtype, cache_dtype, seed=0, tail_rows=0, spare_pages=2, q_scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.csa, self.old, self.new, self.H, self.kv_heads, self.dim = csa, old, new, H, kv_heads, dim
        self.dtype, self.cache_dtype, self.B = dtype, cache_dtype, len(old)
        pages = [-(-(o + n) // PAGE) for o, n in zip(old, new)]
        self.max_pages = max(1, max(pages)) + 1
        order = torch.randperm(sum(pages) + spare_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        table = torch.full((self.B, self.max_pages), -7, dtype=torch.int32)  # ids that must not be read
        for b, p in enumerate(pages):
            table[b, :p] = torch.tensor([order.pop() for _ in range(p)], dtype=torch.int32)
        self.table = table.cuda()
        self.num_pages = sum(pages) + spare_pages
        shape = (self.num_pages, kv_heads, PAGE, dim)
        self.k_pages = torch.full(shape, float("nan"), device="cuda").to(cache_dtype)
        self.v_pages = self.k_pages.clone()
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.n_tokens = torch.tensor(old, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        self.used = sum(new)
        self.total = self.used + tail_rows
        self.max_new = max(new) if new else 0
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        for b, (o, n) in enumerate(zip(old, new)):  # every token that will be held
            at = torch.arange(o + n, device="cuda")
            pg, slot = self.table[b, at // PAGE].long(), at % PAGE
            for pool in (self.k_pages, self.v_pages):
                pool.permute(0, 2, 1, 3)[pg, slot] = rnd(o + n, kv_heads, dim).to(cache_dtype)
        self.q = (rnd(self.total, H, dim) * q_scale).to(dtype)
        self.desc = csa.kv_cache(self.k_pages, self.v_pages, self.table, self.n_tokens, self.status)

    def hold_all(self):
        self.n_tokens.copy_(torch.tensor([o + n for o, n in zip(self.old, self.new)], dtype=torch.int32))

    def attend(self, scale, window=0, q=None, out=None, lse=True, max_new=None, stream=None):
        q = self.q if q is None else q
        out = torch.full_like(self.q, 777.0) if out is None else out
        lse = torch.full((self.total, self.H), 777.0, device="cuda") if lse is True else lse
        mx = self.max_new if max_new is None else max_new
        ws = torch.empty(max(16, self.csa.kv_attn_workspace(self.desc, self.total, mx, self.H)), dtype=torch.uint8, device="cuda")
        ws.fill_(255)  # NaN patterns: nothing may be read before it is written
        self.csa.kv_attn(self.desc, q, self.cu, mx, scale, out, ws, lse=lse, window=window, stream=stream)
        return out, lse

    def check(self, out, lse, scale, window=0, seqs=None, q=None):
        """Compare with the oracle.  Probabilities are rounded once (u_p of each), scores and sums carry fp32 errors,
        the output is rounded once."""
        u_p = 2.0 ** -8 if self.cache_dtype == torch.bfloat16 else 2.0 ** -11
        table = self.table.cpu().numpy()
        kp, vp, qh = host(self.k_pages), host(self.v_pages), host(self.q if q is None else q)
        oh, lh, n_tok = host(out), host(lse) if lse is not None else None, self.n_tokens.cpu().numpy()
        g = self.H // self.kv_heads
        cu = self.cu.cpu().numpy()
        for b in range(self.B) if seqs is None else seqs:
            lo, hi, n = cu[b], cu[b + 1], int(n_tok[b])
            if hi == lo:
                continue
            for h in range(self.kv_heads):
                k, v = okv.rows_of(kp, table, b, n, h), okv.rows_of(vp, table, b, n, h)
                qs = qh[lo:hi, h * g:(h + 1) * g]
                o, l, mag = okv.attention(qs, k, v, n, scale, window)
                # |s| errors: fp32 products and sums of `dim` terms; exp2 and the sums of n terms in fp32
                s_abs = scale * (np.abs(qs) @ np.abs(k).T).max(-1, initial=0.0)[..., None] if n else 0.0
                eps = 2 * (s_abs * self.dim * 2.0 ** -24 + (n / 8 + 64) * 2.0 ** -24)
                got = oh[lo:hi, h * g:(h + 1) * g]
                bound = (u_p + eps) * mag + U[self.dtype] * (np.abs(o) + (u_p + eps) * mag) + TINY[self.dtype] + 1e-30
                bad = ~(np.abs(got - o) <= bound)
                assert not bad.any(), (b, h, np.argwhere(bad)[:4], got[bad][:4], o[bad][:4], bound[bad][:4])
                if lh is not None:
                    gl = lh[lo:hi, h * g:(h + 1) * g]
                    empty = np.isinf(l)
                    assert (np.isneginf(gl) == empty).all()
                    lb = eps[..., 0] if n else 0.0
                    d = np.where(empty, 0.0, np.abs(np.where(empty, 0.0, gl) - np.where(empty, 0.0, l)))
                    assert (d <= lb + 2.0 ** -23 * np.abs(np.where(empty, 0.0, l))).all(), (b, h, d.max())
