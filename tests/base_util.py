"""Inputs, calls and error bounds for the tests of the 4-bit base product and the
gated feed-forward product."""
import numpy as np
import torch

import segmented_gathered_rank_amd as sgr
from oracle import base_oracle as bo

ACT = {"silu": sgr.LORA_ACT_SILU, "gelu": sgr.LORA_ACT_GELU, "gelu_tanh": sgr.LORA_ACT_GELU_TANH}
SENTINEL = -77.0     # exactly representable in bf16


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16()


class Problem:
    """One call's inputs on the GPU and their exact values on the host.

    kind: bf16, fp8, int4, int4z or table.  pads: extra elements per row of x, y, the codes (in
    units of 16 bytes) and the scales (in units of 4)."""

    def __init__(self, op, kind, n, h_in, h_out, page=64, group=64, ranks=(16,), act="silu", ids="random", pads=0,
                 seed=0, load=None, x=None, w_scale=0.05):
        rng = np.random.default_rng(seed)
        self.w_scale = w_scale
        self.op, self.kind, self.n, self.h_in, self.h_out, self.group, self.act = op, kind, n, h_in, h_out, group, act
        self.np = 2 if op == "glu" else 1
        self.ld_x, self.ld_y = h_in + 8 * pads, h_out + 4 * pads
        xv = rng.normal(size=(n, h_in)) if x is None else x
        xb = torch.full((n, self.ld_x), float("nan"), dtype=torch.bfloat16)
        xb[:, :h_in] = bf16(xv)
        self.x64 = xb[:, :h_in].double().numpy()
        self.x = xb.cuda()
        # the rows after the last token and the columns after h_out must stay as they are
        self.y = torch.full((n + 3, self.ld_y), SENTINEL, dtype=torch.bfloat16, device="cuda")
        self.slots = len(ranks)
        self.w64, self.wdev, self.wabs = [], [], []
        for p in range(self.np):
            self._weights(rng, pads)
        self.pool = sgr.lora_pool_create(0, sgr.LORA_BF16, page, 2 * sum(ranks) * (h_in + h_out) // page + 8,
                                         self.slots, 2, [h_in] * 2, [h_out] * 2, max(max(ranks), 1))
        self.adapters = [[None] * self.slots for _ in range(2)]
        for s, r in enumerate(ranks):
            for p in range(2):
                if r == 0 or (load is not None and not load(s, p)):
                    continue
                a, b = bf16(rng.normal(size=(r, h_in)) * 0.05), bf16(rng.normal(size=(r, h_out)) * 0.05)
                sc = float(np.float32(32.0 / r * (1 + 0.25 * p)))
                sgr.lora_pool_load(self.pool, s, p, r, a, b, sc)
                self.adapters[p][s] = (sc, a.double().numpy(), b.double().numpy())
        if isinstance(ids, str):
            ids = {"random": lambda: rng.integers(-1, self.slots, n), "none": lambda: np.full(n, -1),
                   "bad": lambda: rng.integers(-5, self.slots + 5, n),
                   "runs": lambda: np.repeat(rng.integers(-1, self.slots, n), 37)[:n],
                   "one": lambda: np.zeros(n), "null": lambda: None}[ids]()
        self.ids64 = None if ids is None else np.asarray(ids, np.int64)
        self.ids = None if ids is None else torch.from_numpy(self.ids64.astype(np.int32)).cuda()
        nb = sgr.lora_fused_workspace_bytes(self.pool, 0, self.np, n)
        # a workspace of exactly the size asked for, full of NaN
        self.ws = torch.full((max(nb, 16) // 4,), float("nan"), device="cuda")

    def _weights(self, rng, pads):
        kind, h_in, h_out = self.kind, self.h_in, self.h_out
        if kind == "bf16":
            self.ld_w = h_in + 8 * pads
            w = torch.full((h_out, self.ld_w), float("nan"), dtype=torch.bfloat16)
            w[:, :h_in] = bf16(rng.normal(size=(h_out, h_in)) * self.w_scale)
            self.wdev.append(w.cuda())
            self.w64.append(w[:, :h_in].double().numpy().T)
            self.wabs.append(np.abs(self.w64[-1]))
        elif kind == "fp8":
            self.ld_w = h_in + 16 * pads
            codes = rng.integers(0, 256, (h_out, self.ld_w), dtype=np.uint8)
            codes[(codes & 0x7F) == 0x7F] = 0x38
            codes[:, h_in:] = 0x7F
            scale = (0.001 * rng.uniform(0.5, 2, h_out)).astype(np.float32)
            self.wdev.append((torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda()))
            self.w64.append(bo.widen_fp8(codes[:, :h_in], scale))
            self.wabs.append(np.abs(self.w64[-1]))
        else:
            n_g = h_in // self.group
            codes = rng.integers(0, 256, (h_out, h_in // 2 + 16 * pads + (-(h_in // 2)) % 16), dtype=np.uint8)
            scale = bf16(0.02 * rng.uniform(0.5, 2, (n_g, h_out + 4 * pads)) * rng.choice([-1, 1], (n_g, 1)))
            zero = rng.integers(0, 256 if pads else 16, scale.shape, dtype=np.uint8) if kind == "int4z" else None
            table = bf16(rng.normal(size=16)) if kind == "table" else None
            s64 = scale.double().numpy()[:, :h_out]
            z64 = None if zero is None else zero[:, :h_out]
            t64 = None if table is None else table.double().numpy()
            self.w64.append(bo.widen_w4(codes, s64, self.group, z64, t64))
            # where a zero point joins after the product, s q and s z are summed apart
            zz = np.zeros_like(s64) if table is not None else np.full(s64.shape, 8.0) if zero is None else z64
            q = np.abs(self.w64[-1]) + 2 * np.repeat(np.abs(s64) * zz, self.group, 0)
            self.wabs.append(q)
            dev = [None if t is None else torch.as_tensor(t).cuda() for t in (codes, scale, zero, table)]
            self.wdev.append(sgr.lora_w4_bind(dev[0], dev[1], self.group, zero=dev[2], table=dev[3]))

    def call(self, modules=(0, 1), stream=None, y=None, ws=None, n=None, **over):
        y = self.y if y is None else y
        ws = self.ws if ws is None else ws
        n = self.n if n is None else n
        w = self.wdev
        if self.op == "gemm":
            sgr.lora_fused_gemm_w4(self.pool, modules[0], self.x, self.ld_x, w[0], self.ids, n, y, self.ld_y, ws,
                                   stream=stream)
        elif self.kind == "bf16":
            sgr.lora_fused_glu(self.pool, *modules, self.x, self.ld_x, w[0], w[1], self.ld_w, self.ids, n,
                               ACT[self.act], y, self.ld_y, ws, stream=stream)
        elif self.kind == "fp8":
            sgr.lora_fused_glu_fp8w(self.pool, *modules, self.x, self.ld_x, w[0][0], w[1][0], self.ld_w, w[0][1],
                                    w[1][1], self.ids, n, ACT[self.act], y, self.ld_y, ws, stream=stream)
        else:
            sgr.lora_fused_glu_w4(self.pool, *modules, self.x, self.ld_x, w[0], w[1], self.ids, n, ACT[self.act], y,
                                  self.ld_y, ws, stream=stream)

    def reference(self, modules=(0, 1)):
        """(value, bound) per output.

        Each g and u is a sum of fp32 terms over K = h_in products (and the adapter's): at most
        K + 128 roundings of 2^-24 relative to the sum S of absolute products meet any one term,
        and the tiled path's two-part t adds 2^-16 of the adapter's share of S.  The gate passes an
        error of g on with |act'| <= 1.13 and adds a few fp32 roundings of its own, |act(g)| <= |g|.
        The result is rounded once: half a bf16 step, 2^-8 of the value at most."""
        eps = (self.h_in + 128) * 2.0 ** -24 + 2.0 ** -16
        gs = []
        for p in range(self.np):
            y, s = bo.linear(self.x64, self.w64[p], self.ids64, self.adapters[modules[p]])
            gs.append((y, eps * (s + np.abs(self.x64) @ (self.wabs[p] - np.abs(self.w64[p])))))
        if self.op == "gemm":
            v, e = gs[0]
        else:
            (g, eg), (u, eu) = gs
            a = bo.activation(self.act, g)
            v = a * u
            ea = 1.13 * eg + 2.0 ** -20 * np.abs(g)
            e = ea * np.abs(u) + (np.abs(a) + ea) * eu
        return v, (np.abs(v) + e) * 2.0 ** -8 + e

    def check(self, modules=(0, 1), what=""):
        torch.cuda.synchronize()
        got = self.y.double().cpu().numpy()
        assert np.all(got[self.n:] == SENTINEL) and np.all(got[:, self.h_out:] == SENTINEL), "wrote past the output"
        v, bound = self.reference(modules)
        off = np.abs(got[:self.n, :self.h_out] - v)
        worst = np.max(off / np.maximum(bound, 1e-300)) if off.size else 0.0
        assert np.all(off <= bound), f"{what}: {worst:.2f} times the bound"
        return worst

    def close(self):
        torch.cuda.synchronize()
        sgr.lora_pool_destroy(self.pool)
