"""Shared by the chunk operators' tests: a paged FP8 cache with ragged
sequences, stale bytes (NaN codes, NaN and infinite scales among them)
everywhere that no token lives, and float64 restatements of the definitions."""
from __future__ import annotations

import dataclasses

import torch


def e4m3(codes: torch.Tensor) -> torch.Tensor:
    """OCP E4M3 values of uint8 codes, from the format's definition (float64)."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7).double(), m * 2.0**-9)
    mag = torch.where((c & 127) == 127, float("nan"), mag)
    return torch.where(c >= 128, -mag, mag)


def quantise(x: torch.Tensor):
    """(codes, scales) of bf16 rows by the append's rule, on the CPU in fp32."""
    x = x.float()
    amax = x.abs().amax(-1)
    s = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    return (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s


@dataclasses.dataclass
class Cache:
    """A CPU-side cache and the chunk that is about to arrive."""
    new: list      # new tokens of each sequence
    have: list     # cached tokens of each sequence
    B_k: int
    H_kv: int
    d_h: int
    d_idx: int
    seed: int = 0
    pad: int = 0   # padding rows behind the last sequence
    spare_pages: int = 3

    def __post_init__(self):
        g = torch.Generator().manual_seed(1000 + self.seed)
        self.g = g
        S, B = len(self.new), self.B_k
        self.S, self.T = S, sum(self.new) + self.pad
        need = [(n + h + B - 1) // B for n, h in zip(self.new, self.have)]
        self.max_pages = max(1, max(need)) + 1
        self.n_pages = sum(need) + self.spare_pages
        self.cu = torch.tensor([sum(self.new[:s]) for s in range(S + 1)], dtype=torch.int32)
        self.len = torch.tensor(self.have, dtype=torch.int32)
        order = torch.randperm(self.n_pages, generator=g)
        # entries past a sequence's pages are garbage
        self.table = torch.randint(-5, self.n_pages + 5, (S, self.max_pages), generator=g,
                                   dtype=torch.int32)
        at = 0
        for s in range(S):
            self.table[s, : need[s]] = order[at: at + need[s]].to(torch.int32)
            at += need[s]
        self.pool = {}
        for name, shape in (("k", (self.H_kv, self.d_h)), ("v", (self.H_kv, self.d_h)),
                            ("i", (self.d_idx,))):
            # stale memory: any byte (0x7f and 0xff are NaN), any scale
            codes = torch.randint(0, 256, (self.n_pages, B, *shape), generator=g, dtype=torch.uint8)
            scale = torch.randn(self.n_pages, B, *shape[:-1], generator=g)
            pick = torch.randint(0, 6, scale.shape, generator=g)
            scale = torch.where(pick == 0, float("nan"), torch.where(pick == 1, float("inf"), scale))
            self.pool[name] = [codes, scale]
        self.dense = {}  # per sequence float64 rows of all positions, cached and new
        self.rows = {n: torch.zeros(self.T, *sh, dtype=torch.bfloat16) for n, sh in
                     (("k", (self.H_kv, self.d_h)), ("v", (self.H_kv, self.d_h)), ("i", (self.d_idx,)))}
        for s in range(S):
            n, h = self.new[s], self.have[s]
            for name in ("k", "v", "i"):
                shape = self.rows[name].shape[1:]
                x = torch.randn(h + n, *shape, generator=g).bfloat16()
                x[::7] *= 0.01  # scales differ from token to token
                self.rows[name][self.cu[s]: self.cu[s + 1]] = x[h:]
                codes, scale = quantise(x)
                self.dense[s, name] = e4m3(codes) * scale.double()[..., None]
                page, slot = self.where(s, torch.arange(h))
                self.pool[name][0][page, slot] = codes[:h]
                self.pool[name][1][page, slot] = scale[:h]

    def where(self, s, positions):
        return self.table[s].long()[positions // self.B_k], positions % self.B_k

    def positions(self):
        pos = torch.full((self.T,), -1, dtype=torch.int32)
        for s in range(self.S):
            pos[self.cu[s]: self.cu[s + 1]] = self.have[s] + torch.arange(self.new[s], dtype=torch.int32)
        return pos

    def appended(self):
        """The pools after the append: {name: [codes, scales]}."""
        out = {n: [t.clone() for t in p] for n, p in self.pool.items()}
        for s in range(self.S):
            page, slot = self.where(s, self.have[s] + torch.arange(self.new[s]))
            for name in out:
                codes, scale = quantise(self.rows[name][self.cu[s]: self.cu[s + 1]])
                out[name][0][page, slot], out[name][1][page, slot] = codes, scale
        return out

    def gpu(self, pools=None):
        """Device tensors in the order of the entry points' arguments."""
        p = pools or self.pool
        d = {n + e: p[n][j].cuda() for n in p for j, e in enumerate(("p", "s"))}
        d.update(table=self.table.cuda(), cu=self.cu.cuda(), len=self.len.cuda(),
                 **{"new_" + n: r.cuda() for n, r in self.rows.items()})
        return d

    def pools(self, d):
        return d["kp"], d["ks"], d["vp"], d["vs"], d["ip"], d["is"]
