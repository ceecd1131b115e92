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
    wide: int = 0  # page-table entries per sequence, when more than needed

    def __post_init__(self):
        g = torch.Generator().manual_seed(1000 + self.seed)
        self.g = g
        S, B = len(self.new), self.B_k
        self.S, self.T = S, sum(self.new) + self.pad
        need = [(n + h + B - 1) // B for n, h in zip(self.new, self.have)]
        self.max_pages = max(max(need) + 1, self.wide)
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


def refresh(c: Cache) -> None:
    """Recompute the dense rows of the new tokens after c.rows was changed."""
    for s in range(c.S):
        for name in ("k", "v", "i"):
            codes, scale = quantise(c.rows[name][c.cu[s]: c.cu[s + 1]])
            c.dense[s, name][c.have[s]:] = e4m3(codes) * scale.double()[..., None]


def selection(c: Cache, k: int, holes: bool = False) -> torch.Tensor:
    """Random selections [T, H_kv, k]: the own block and earlier ones, ascending,
    -1 padded; with `holes`, also empty rows, blocks after the row's own and
    rows without their own block."""
    idx = torch.full((c.T, c.H_kv, k), -1, dtype=torch.int32)
    pos = c.positions()
    for t in range(c.T):
        own = int(pos[t]) // c.B_k if pos[t] >= 0 else 0
        for h in range(c.H_kv):
            pick = torch.randperm(own, generator=c.g)[: k - 1].tolist() + [own]
            if holes:
                kind = (t + h) % 5
                if kind == 1:
                    pick = []
                elif kind == 2:
                    pick = pick[:-1]
                elif kind == 3 and own + 1 < c.max_pages and len(pick) < k:
                    pick = pick + [own + 1]
            pick = sorted(pick)
            idx[t, h, : len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return idx


def attention(c: Cache, q, idx, scale):
    """(o, lse, tolerances of both) in float64.

    Rounding of the kernels: o is rounded to bf16 once (2^-8 of it); a weight
    times its value's scale is rounded to 11 bits, or to 2^-25 of the largest
    one; n products are added in fp32 (a unit of the last place, 2^-23, each);
    an error of a score enters its weight and the sum of weights."""
    T, H_q, d = q.shape
    G = H_q // c.H_kv
    o = torch.zeros(T, H_q, d, dtype=torch.float64)
    lse = torch.full((T, H_q), -float("inf"), dtype=torch.float64)
    otol, ltol = torch.zeros_like(o), torch.zeros(T, H_q, dtype=torch.float64)
    pos = c.positions()
    for s in range(c.S):
        for t in range(int(c.cu[s]), int(c.cu[s + 1])):
            for h in range(c.H_kv):
                j = [torch.arange(b * c.B_k, min((b + 1) * c.B_k, int(pos[t]) + 1))
                     for b in idx[t, h].tolist() if 0 <= b <= int(pos[t]) // c.B_k]
                j = torch.cat(j) if j else torch.zeros(0, dtype=torch.long)
                if not len(j):
                    continue
                K, V = c.dense[s, "k"][j, h], c.dense[s, "v"][j, h]
                rows = slice(h * G, (h + 1) * G)
                x = q[t, rows].double() @ K.T * scale
                err = (q[t, rows].double().abs() @ K.abs().T * scale * (d * 2.0**-23 + 2.0**-20)).amax(-1)
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - z[:, None])
                o[t, rows], lse[t, rows] = w @ V, z
                n = len(j)
                mag = w @ V.abs()
                rel = 2.0**-11 + n * 2.0**-23 + 2 * err[:, None] + 2.0**-18
                big = (w[..., None] * V.abs()[None]).amax((1, 2)) if V.numel() else 0.0
                # the largest weight times scale, times any code, is at most 448 times that scale
                otol[t, rows] = o[t, rows].abs() * 2.0**-8 + rel * mag + (n * 2.0**-25 * big)[:, None]
                ltol[t, rows] = err + 2.0**-18 + z.abs() * 2.0**-21
    return o, lse, otol, ltol
