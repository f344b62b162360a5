"""Inputs and 64-bit statements shared by the tests of the operators around the
paged cache."""
import numpy as np
import torch

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "int8": torch.int8}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def f64(t):
    """A tensor's values on the host in 64 bits."""
    t = t.float() if t.dtype == torch.float8_e4m3fn else t
    return t.double().cpu().numpy()


def on_gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


class Cache:
    """A pool of random contents behind a shuffled table.  ``poison`` fills every row
    that no sequence owns (and page 0, which none owns) with NaN, so that a read past a
    length or through an absent page shows."""

    def __init__(self, lens, kind, hkv, d, ps, seed=0, extra_cols=0, poison=True, drop=(),
                 free_scales=False):
        rng = np.random.default_rng(seed)
        self.lens, self.kind, self.hkv, self.d, self.ps = [max(int(n), 0) for n in lens], kind, hkv, d, ps
        live = [-(-n // ps) for n in self.lens]
        cols = max(max(live), 1) + extra_cols
        n = sum(live) + 2
        ids = 1 + rng.permutation(n - 1).astype(np.int32)
        self.bt = np.full((len(lens), cols), -1, np.int32)
        at = 0
        for b, m in enumerate(live):
            self.bt[b, :m] = ids[at:at + m]
            at += m
        for b, c in drop:
            self.bt[b, c] = -1
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.eight = kind in ("e4m3", "int8")
        self.pages, self.scales = [], []
        for _ in range(2):
            x = torch.randn((n, hkv, ps, d), generator=gen, device="cuda")
            if kind == "int8":
                x = (x * 40).round().clamp(-127, 127)
            elif kind == "e4m3":
                x = (x * 100).clamp(-448, 448)
            self.pages.append(x.to(TORCH[kind]))
            s = None
            if self.eight:
                s = 2.0 ** rng.integers(-9, -4, (n, hkv)).astype(np.float64)
                if free_scales:
                    s = s * rng.uniform(1, 2, s.shape)
                s = on_gpu(s, np.float32)
            self.scales.append(s)
        self.table = on_gpu(self.bt, np.int32)
        self.used = on_gpu(np.asarray(lens), np.int32)
        # what stands for the values: taken before rows that nothing owns are spoilt
        self.values = []
        for p, s in zip(self.pages, self.scales):
            v = f64(p)
            if s is not None:
                v = v * f64(s)[:, :, None, None]
            self.values.append(v)
        if poison:
            owned = torch.zeros((n, ps), dtype=torch.bool)
            for b, m in enumerate(self.lens):
                for c in range(min(-(-m // ps), cols)):
                    if self.bt[b, c] >= 0:
                        owned[self.bt[b, c], :min(ps, m - c * ps)] = True
            dead = (~owned).cuda()[:, None, :, None]
            for i, p in enumerate(self.pages):
                if kind == "int8":
                    self.pages[i] = torch.where(dead, torch.full_like(p, -128), p)
                elif kind == "e4m3":
                    bits = p.view(torch.uint8)
                    self.pages[i] = torch.where(dead, torch.full_like(bits, 0x7F), bits).view(p.dtype)
                else:
                    self.pages[i] = torch.where(dead, torch.full_like(p, float("nan")), p)
            if self.eight:
                gone = (~owned.any(1)).cuda()[:, None]
                self.scales = [torch.where(gone, torch.full_like(s, float("nan")), s)
                               for s in self.scales]

    def kw(self):
        return dict(k_scales=self.scales[0], v_scales=self.scales[1]) if self.eight else {}

    def v_scales(self, b, positions):
        """V's scales [n, hkv] at positions of sequence b (1 for the wider types)."""
        out = np.ones((len(positions), self.hkv))
        if self.eight:
            s = f64(self.scales[1])
            for i, p in enumerate(positions):
                out[i] = s[max(self.bt[b, p // self.ps], 0)]
        return out

    def rows(self, b, positions, which):
        """Values [n, hkv, d] of positions of sequence b (zeros where there is no page),
        and which of them exist."""
        out = np.zeros((len(positions), self.hkv, self.d))
        there = np.zeros(len(positions), bool)
        for i, p in enumerate(positions):
            c = p // self.ps
            if 0 <= p < self.lens[b] and c < self.bt.shape[1] and 0 <= self.bt[b, c]:
                out[i] = self.values[which][self.bt[b, c], :, p % self.ps]
                there[i] = True
        return out, there
