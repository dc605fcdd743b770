"""Plain references of the key-value cache's operators in 64 bits (CPU), and the
batches that their tests use."""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def page_values(x):
    """x [P, D] of one head's full page, float64 -> the float32 numbers that its codes stand for."""
    x = x.astype(np.float32)
    if not np.isfinite(x).all():
        return np.full(x.shape, np.nan, np.float32)
    top = np.abs(x).max()
    if top < np.float32(2.0 ** -119):
        return np.zeros(x.shape, np.float32)
    inv, scale = np.float32(127.0) / top, top / np.float32(127.0)
    return (np.rint(x * inv) * scale).astype(np.float32)


def held_values(x, P):
    """x [n, heads, D]: all tokens of a sequence (torch) -> what the cache holds of them, float32."""
    y = x.detach().float().cpu().numpy().copy()
    n, heads, _ = y.shape
    for h in range(heads):
        for p in range(n // P):
            y[p * P:(p + 1) * P, h] = page_values(y[p * P:(p + 1) * P, h])
        for t in range(n // P * P, n):
            if not np.isfinite(y[t, h]).all():
                y[t, h] = np.nan
    return torch.from_numpy(y)


def attention(q, k, v, first, scale, window=0, hidden=None):
    """q [n, heads, D] at positions first .., k, v [total, kv heads, D] (any float), hidden: keys that nobody sees
    -> out float64 [n, heads, D] and how far a result of the kernel's type of arithmetic may be from it before its
    last rounding, the same shape.

    The kernel's sums, maxima and exponentials are binary32, its products exact in binary32 up to that, a weight
    is rounded to fp16 as a multiple of 2^-11 of the largest that there can be: by relative 2^-11, or, among fp16's
    subnormal numbers (steps of 2^-24), by half of 2^-24 2^-11 = 2^-36 of the largest.  A sum of n terms is off by at most n 2^-23 of the sum of magnitudes, a score by D 2^-23 of its
    products' magnitudes, and 8 more roundings on the way."""
    q, k, v = (t.detach().double().cpu() for t in (q, k, v))
    n, heads, D = q.shape
    total, kv = k.shape[0], k.shape[1]
    G = heads // kv
    out, far = torch.zeros_like(q), torch.zeros_like(q)
    pos = first + torch.arange(n)[:, None]
    j = torch.arange(total)
    seen = j <= pos
    if window:
        seen = seen & (j > pos - window)
    if hidden is not None:
        seen = seen & ~hidden
    for h in range(heads):
        kk, vv = k[:, h // G], v[:, h // G]
        # what is out of sight has no part, whatever it is
        s = torch.zeros((n, total), dtype=torch.float64)
        size = torch.zeros_like(s)
        some = seen.any(0).nonzero()[:, 0]
        s[:, some] = q[:, h] @ kk[some].t() * scale
        size[:, some] = q[:, h].abs() @ kk[some].abs().t() * abs(scale)
        s = torch.where(seen, s, -math.inf)
        top = s.amax(1, keepdim=True)
        p = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
        z = p.sum(1, keepdim=True)
        p = p / torch.where(z == 0, 1.0, z)
        # (a value that is NaN is one for those who see it only: 0 times NaN is not formed)
        lost = (seen[:, some].double() @ torch.isnan(vv[some]).double()) > 0
        vv = torch.nan_to_num(vv)
        out[:, h] = torch.where(lost, math.nan, p[:, some] @ vv[some])
        size = torch.where(seen, size, 0.0).amax(1, keepdim=True)
        delta = (D + 8) * 2.0 ** -23 * size + 2.0 ** -22
        mass = p[:, some] @ vv[some].abs()
        most = vv[some].abs().amax(0, keepdim=True) if some.numel() else 0.0
        far[:, h] = (2.0 ** -11 + 2.1 * delta + (total + 16) * 2.0 ** -23) * mass + total * 2.0 ** -36 * most
    return out, far


def check(got, want, far):
    """got (bf16 or f16) against want, within far and the rounding of its type."""
    got64 = got.detach().double().cpu()
    assert torch.equal(torch.isnan(got64), torch.isnan(want)), "NaN elsewhere than in the reference"
    ok = ~torch.isnan(want)
    half = HALF[got.dtype]
    room = far + half * (want.abs() + far) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    assert torch.isfinite(room[ok]).all()
    bad = ((got64 - want).abs() > room) & ok
    assert not bad.any(), (int(bad.sum()), ((got64 - want).abs() / room)[ok].max().item(), bad.nonzero()[0].tolist())


class Batch:
    """Sequences of `held` tokens that get `new` ones, their pages scattered, their slots out of order; the tokens'
    keys and values, all of them and the call's."""

    def __init__(self, held, new, kv, D, P, dtype=torch.bfloat16, seed=0, spare=2, device="cuda", scale=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.held, self.new, self.P, self.dtype, self.device = list(held), list(new), P, dtype, device
        self.kv, self.D = kv, D
        B = len(held)
        need = [-(-(h + n) // P) for h, n in zip(held, new)]
        width = max(max(need), 1) + spare
        ids = torch.randperm(sum(need) + 3, generator=gen, dtype=torch.int32)
        self.pages = ids.numel()
        self.table_cpu = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table_cpu[i, :n] = ids[at:at + n]
            at += n
        self.slots_cpu = torch.randperm(B + 2, generator=gen, dtype=torch.int32)[:B].contiguous()

        def tokens():
            spread = torch.exp(0.5 * torch.randn((kv, D), generator=gen))
            return [(scale * spread * torch.randn((h + n, kv, D), generator=gen)).to(dtype) for h, n in zip(held, new)]

        self.k_all, self.v_all = tokens(), tokens()
        self.gen = gen

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.device)

    def args(self, held=None, new=None):
        """table, lens, slots, cu of the step that adds `new` tokens to `held` ones."""
        held = self.held if held is None else held
        new = self.new if new is None else new
        return (self.table_cpu.to(self.device), self.ints(held), self.slots_cpu.to(self.device),
                self.ints([0, *np.cumsum(new).tolist()]))

    def cut(self, x, held, new):
        """The tokens of a step out of all, on the device."""
        return torch.cat([t[h:h + n] for t, h, n in zip(x, held, new)]).to(self.device)

    def cache(self, binding, filled=True):
        """A cache that holds the sequences' held tokens."""
        c = binding.KvCache(self.pages, len(self.held) + 2, self.kv, self.D, page_size=self.P, device=self.device)
        if filled and sum(self.held):
            zero = [0] * len(self.held)
            table, lens, slots, cu = self.args(zero, self.held)
            binding.kv_append(c, self.cut(self.k_all, zero, self.held), self.cut(self.v_all, zero, self.held), table,
                              lens, slots, cu=cu)
        return c

    def append_new(self, binding, cache):
        table, lens, slots, cu = self.args()
        binding.kv_append(cache, self.cut(self.k_all, self.held, self.new), self.cut(self.v_all, self.held, self.new),
                          table, lens, slots, cu=cu)

    def queries(self, heads, scale=1.0):
        return (scale * torch.randn((sum(self.new), heads, self.D), generator=self.gen)).to(self.dtype).to(self.device)

    def attention(self, q, scale=None, window=0, hidden=None):
        """Reference and room of the step's attention."""
        scale = self.D ** -0.5 if scale is None else scale
        outs, fars, at = [], [], 0
        for i, (h, n) in enumerate(zip(self.held, self.new)):
            if n == 0:
                continue
            o, f = attention(q[at:at + n], held_values(self.k_all[i], self.P), held_values(self.v_all[i], self.P), h,
                             scale, window, None if hidden is None else hidden[i])
            outs.append(o)
            fars.append(f)
            at += n
        return torch.cat(outs), torch.cat(fars)
