"""Problems on the paged key/value cache, and what the operators must return for them, in 64 bits.

Everything is plain torch on whatever device the problem lives on; no code is shared with the library."""

from __future__ import annotations

import math

import torch

import block_quantized_matmul_lwq_b200 as lwq

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Problem:
    """A cache with shuffled pages, B sequences of ``lens`` tokens (``new`` of them new), an optional prefix.

    Pages that no live token needs, and the rest of each last page, hold NaN: nothing may read them into a result."""

    def __init__(self, dev, dtype, lens, H, Hkv, D, page, new=None, prefix=0, spare=3, seed=0, max_pages=None,
                 poison=True):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        self.dev, self.dtype, self.H, self.Hkv, self.D, self.page = dev, dtype, H, Hkv, D, page
        self.lens, self.new, self.prefix = list(lens), list(new or [1] * len(lens)), prefix
        self.B, self.T = len(self.lens), sum(self.new)
        self.G = H // Hkv
        t = TYPES[dtype]
        need = [-(-max(n, 0) // page) for n in self.lens]
        npre = -(-prefix // page)
        self.max_pages = max_pages or max(1, max(need))
        self.num_pages = sum(need) + npre + spare
        perm = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        self.tables_h = torch.full((self.B, self.max_pages), -7, dtype=torch.int32)   # unread entries: no page
        at = npre
        for b, k in enumerate(need):
            self.tables_h[b, :k] = perm[at:at + k]
            at += k
        self.prefix_h = perm[:npre].clone()
        shape = (self.num_pages, Hkv, page, D)
        self.kc = torch.randn(shape, generator=g).to(t).to(dev)
        self.vc = torch.randn(shape, generator=g).to(t).to(dev)
        if poison:
            live = torch.zeros(self.num_pages, page, dtype=torch.bool)
            for b, n in enumerate(self.lens):
                for j in range(max(n, 0)):
                    live[self.tables_h[b, j // page], j % page] = True
            for j in range(prefix):
                live[self.prefix_h[j // page], j % page] = True
            dead = ~live.to(dev)
            self.kc.transpose(1, 2)[dead] = float("nan")
            self.vc.transpose(1, 2)[dead] = float("nan")
        self.tables, self.prefix_pages = self.tables_h.to(dev), self.prefix_h.to(dev)
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        cu = [0]
        for n in self.new:
            cu.append(cu[-1] + n)
        self.cu = cu
        self.cu_d = torch.tensor(cu, dtype=torch.int32, device=dev)
        self.q = torch.randn((self.T, H, D), generator=g).to(t).to(dev)
        self.scale = D ** -0.5

    def cache(self) -> lwq.lwq_paged:
        return lwq.lwq_paged(lwq.ACT_DTYPES[self.dtype], self.kc, self.vc, self.tables, self.lens_d, B=self.B,
                             Hkv=self.Hkv, D=self.D, page=self.page, max_pages=self.max_pages,
                             num_pages=self.num_pages, prefix=self.prefix_pages if self.prefix else None,
                             prefix_len=self.prefix)

    def rows(self, b, n):
        """K and V of the prefix and the first n tokens of sequence b, [Hkv][prefix + n][D] in 64 bits."""
        j = torch.arange(max(n, 0))
        pages = torch.cat([self.prefix_h[torch.arange(self.prefix) // self.page],
                           self.tables_h[b][j // self.page]]).long().to(self.dev)
        offs = torch.cat([torch.arange(self.prefix) % self.page, j % self.page]).to(self.dev)
        k = self.kc[pages, :, offs].double().transpose(0, 1)
        v = self.vc[pages, :, offs].double().transpose(0, 1)
        return k, v

    def expected(self, causal):
        """(out, den, smax): outputs [T][H][D], sum_j p_j |v_j| beside them, and the largest
        scale * sum_i |q_i k_ij| of any score, which bounds the scores' rounding."""
        out = torch.zeros((self.T, self.H, self.D), dtype=torch.float64, device=self.dev)
        den = torch.zeros_like(out)
        smax = 0.0
        cap = self.max_pages * self.page
        for b in range(self.B):
            for i in range(self.new[b]):
                t = self.cu[b] + i
                place = self.lens[b] - self.new[b] + i
                n = place + 1 if causal else self.lens[b]
                if causal and place < 0:
                    continue
                k, v = self.rows(b, min(max(n, 0), cap))
                if k.shape[1] == 0:
                    continue
                q = self.q[t].double().view(self.Hkv, self.G, self.D)
                s = torch.einsum("hgd,hnd->hgn", q, k) * self.scale
                w = torch.softmax(s, -1)
                out[t] = torch.einsum("hgn,hnd->hgd", w, v).reshape(self.H, self.D)
                den[t] = torch.einsum("hgn,hnd->hgd", w, v.abs()).reshape(self.H, self.D)
                smax = max(smax, float((torch.einsum("hgd,hnd->hgn", q.abs(), k.abs()) * abs(self.scale)).max()))
        return out, den, smax


def attention_bound(p: Problem, smax: float, out16: bool) -> float:
    """Largest |out - exact| / sum_j p_j |v_j|.

    Scores: D products summed in 32 bits, each addition off by at most 2^-23 of the sum of magnitudes (tensor
    cores may truncate), so a score is off by D 2^-23 smax and a weight by as much relative to itself; twice, for
    the sum in the denominator.  Exponentials and the scaling into powers of two: 2^-21 of a score's magnitude,
    and 2^-21.  The weighted sum over n keys: (n / 16 + 64) additions of 2^-23.  Weights: kept to 16 bits in two
    bf16 parts, or rounded once to the cache's type when out has that type, whose own rounding comes on top."""
    n = p.prefix + max(max(p.lens), 0)
    eps = torch.finfo(TYPES[p.dtype]).eps / 2
    bound = 2 * (p.D * 2.0 ** -23 + 2.0 ** -21) * smax + 2.0 ** -20 + 2 * (n / 16 + 64) * 2.0 ** -23
    return bound + (2 * eps if out16 else 2.0 ** -16)


def check_attention(p: Problem, causal: bool, out16=False, stream=None):
    t = TYPES[p.dtype] if out16 else torch.float32
    out = torch.full((p.T, p.H, p.D), float("nan"), dtype=t, device=p.dev)
    flags = lwq.LWQ_FLAG_OUT16 if out16 else 0
    if causal:
        lwq.lwq_attention_prefill(p.cache(), p.q, out, p.cu_d, p.T, p.H, p.scale, flags=flags, stream=stream)
    else:
        lwq.lwq_attention_paged(p.cache(), p.q, out, p.H, p.scale, flags=flags, stream=stream)
    torch.cuda.synchronize(p.dev)
    assert_attention(p, out, causal, out16)
    return out


def assert_attention(p: Problem, out, causal: bool, out16=False):
    ref, den, smax = p.expected(causal)
    assert torch.isfinite(out).all()
    zero = den == 0
    assert (out[zero] == 0).all()
    tiny = torch.finfo(out.dtype).tiny          # 16-bit results below the normal range round to multiples of it
    err = ((out.double() - ref).abs() - tiny).clamp_min(0) / torch.where(zero, torch.ones_like(den), den)
    bound = attention_bound(p, smax, out16)
    worst = float(err[~zero].max()) if (~zero).any() else 0.0
    assert worst <= bound, f"error {worst:.3e} > {bound:.3e}"
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK


# ------------------------------------------------------------------- append
def rotate64(x, pos, rot, layout, base=None, inv_freq=None, sections=None):
    """x [T][heads][D] in 64 bits, pos [axes][T] -> rotated."""
    half = rot // 2
    freq = [base ** (-2.0 * i / rot) for i in range(half)] if inv_freq is None else [float(f) for f in inv_freq]
    axis = [a for a, n in enumerate(sections or [half]) for _ in range(n)]
    out = x.clone()
    for i in range(half):
        # positions below 2^31 times a double: reduce in exact rational arithmetic per frequency
        ang = torch.tensor([_angle(int(p), freq[i]) for p in pos[axis[i]].tolist()], dtype=torch.float64,
                           device=x.device)[:, None]
        a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = torch.cos(ang), torch.sin(ang)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


_TWO_PI = None


def _angle(p: int, f: float) -> float:
    """p * f modulo 2 pi, the product taken exactly and 2 pi to 60 digits."""
    global _TWO_PI
    from fractions import Fraction
    if _TWO_PI is None:
        _TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
    x = Fraction(f) * p
    return float(x - _TWO_PI * math.floor(x / _TWO_PI))


def append_inputs(p: Problem, src: str, seed=1, fused=True):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    n = (p.H + 2 * p.Hkv) * p.D
    x = torch.randn((p.T, n), generator=g).to(TYPES[src]).to(p.dev)
    return x, n


def expected_append(p: Problem, x, pos, rope_args, T=None):
    """(q_out, k rows, v rows, bound of their errors) of the T tokens in 64 bits."""
    y = x.double().view(x.shape[0], p.H + 2 * p.Hkv, p.D)
    q, k, v = y[:, :p.H], y[:, p.H:p.H + p.Hkv], y[:, p.H + p.Hkv:]
    if rope_args is None:
        return q, k, v
    qk = rotate64(y[:, :p.H + p.Hkv], pos, **rope_args)
    return qk[:, :p.H], qk[:, p.H:], v
