"""The base products under the adapters whose weights are 4-bit codes, and the
gated feed-forward product: the cases that stand for them, their plain forms,
and the library's calls.

A case names the operator ("gemm": y = x W + adapter term; "glu":
h = act(x Wg + term) * (x Wu + term)), what the base weights are stored as
("bf16", "fp8", or 4-bit codes: "int4" with the zero point 8, "int4z" with a
zero point per group, "table" with a 16-entry codebook), the widths, the batch
and its adapters.
"""
import math

import torch

own = False

DEV = "cuda"
ACTS = ("silu", "gelu", "gelu_tanh")
MIXED_RANKS = (8, 16, 32, 64)


def _case(name, op, kind, n, h_in, h_out, page, slots, rank, run, act="silu", group=0, adapters=True):
    return {"name": name, "op": op, "kind": kind, "n": n, "h_in": h_in, "h_out": h_out, "page": page,
            "slots": slots, "rank": rank, "run": run, "act": act, "group": group, "adapters": adapters}


def listed():
    return [
        # one sequence being decoded, on the small square layer of an encoder: launch latency is all of it
        _case("w4 1 token 768", "gemm", "int4", 1, 768, 768, 768, 8, 16, 1, group=128),
        # one sequence being decoded with its adapter, on a 4096-wide projection
        _case("w4 1 token 4096", "gemm", "int4", 1, 4096, 4096, 4096, 32, 16, 1, group=128),
        # a decode batch in which most tokens bring an adapter of their own, codebook weights
        _case("w4 table 64 tokens", "gemm", "table", 64, 4096, 4096, 4096, 32, 16, 1, group=64),
        # a wide layer without adapters, one token: the weights' read is all of it
        _case("w4 1 token wide", "gemm", "int4z", 1, 8192, 28672, 4096, 1, 16, 1, group=128, adapters=False),
        # decode tokens beside one short prompt: odd widths, small groups, mixed ranks
        _case("w4 177 tokens odd", "gemm", "int4z", 177, 4160, 5440, 320, 64, 0, 29, group=32),
        # a prefill of several prompts, one adapter each
        _case("w4 prefill", "gemm", "int4", 4096, 4096, 4096, 4096, 8, 16, 512, group=128),
        # one sequence being decoded through a gated block
        _case("glu bf16 1 token", "glu", "bf16", 1, 4096, 11264, 1024, 32, 16, 1),
        # a decode batch through a gated block of 4-bit weights
        _case("glu w4 33 tokens", "glu", "int4z", 33, 4096, 12288, 4096, 32, 16, 1, group=128),
        # a decode batch through a gated block of 8-bit weights, mixed ranks
        _case("glu fp8 64 tokens", "glu", "fp8", 64, 2048, 8192, 2048, 64, 0, 1, act="gelu"),
        # an encoder's batch of short sequences: ragged rows, many adapters
        _case("glu table 1000 tokens", "glu", "table", 1000, 768, 2304, 768, 64, 16, 128, act="gelu_tanh", group=64),
        # the same prefill through a gated block of 8-bit weights
        _case("glu fp8 prefill", "glu", "fp8", 2111, 4096, 8192, 4096, 8, 16, 300),
        # the largest: a full prefill through a gated block
        _case("glu bf16 prefill", "glu", "bf16", 4096, 4096, 12288, 4096, 8, 16, 512),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = 4096 * 4096 * 12288 * 2
    while True:
        op = rng.choice(("gemm", "glu"))
        kind = rng.choice(("int4", "int4z", "table") if op == "gemm" else ("bf16", "fp8", "int4", "int4z", "table"))
        page = 64 * log(1, 32)
        h_in = page * rng.randint(1, 32)
        h_out = page * rng.randint(1, 64)
        if not (512 <= h_in <= 12288 and 512 <= h_out <= 28672):
            continue
        n = log(1, 4096)
        if n * h_in * h_out * (2 if op == "glu" else 1) > most // 2:
            continue
        groups = [g for g in (32, 64, 128) if h_in % g == 0]
        return {"op": op, "kind": kind, "n": n, "h_in": h_in, "h_out": h_out, "page": page,
                "slots": log(1, 64), "rank": rng.choice((0, 4, 16, 17, 64)), "run": log(1, 512) if n > 64 else 1,
                "act": rng.choice(ACTS), "group": rng.choice(groups) if kind in ("int4", "int4z", "table") else 0,
                "adapters": rng.random() < 0.85}


def _ranks(case):
    if case["rank"]:
        return [case["rank"]] * case["slots"]
    return [MIXED_RANKS[s % 4] for s in range(case["slots"])]


def _projections(case):
    return 2 if case["op"] == "glu" else 1


# ------------------------------------------------------------------ inputs
def _weights(case, g):
    """One projection's base weights as a layer stores them: [h_out][h_in], spread about 0.02."""
    kind, h_in, h_out = case["kind"], case["h_in"], case["h_out"]
    if kind == "bf16":
        return {"w": (torch.randn(h_out, h_in, device=DEV, generator=g) * 0.02).bfloat16()}
    if kind == "fp8":
        w = torch.randn(h_out, h_in, device=DEV, generator=g) * 0.02
        scale = w.abs().amax(1) / 448
        return {"codes": (w / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), "scale": scale}
    n_g = h_in // case["group"]
    table = zero = None
    if kind == "table":   # the 16 quantile midpoints of a normal, largest value 1
        q = torch.special.ndtri((torch.arange(16, dtype=torch.float64) + 0.5) / 16)
        table = (q / q[-1]).to(torch.bfloat16).to(DEV)
        codes = torch.randint(0, 16, (h_out, h_in), device=DEV, generator=g, dtype=torch.uint8)
        scale = 0.037 * (0.75 + 0.5 * torch.rand(n_g, h_out, device=DEV, generator=g))
    else:
        z = 8.0
        if kind == "int4z":
            zero = torch.randint(5, 11, (n_g, h_out), device=DEV, generator=g, dtype=torch.uint8)
            z = zero.t().float().repeat_interleave(case["group"], 1)
        w = torch.randn(h_out, h_in, device=DEV, generator=g) * 2.7
        codes = (w + z).round().clamp(0, 15).to(torch.uint8)
        scale = 0.0074 * (0.75 + 0.5 * torch.rand(n_g, h_out, device=DEV, generator=g))
    return {"codes": codes[:, 0::2] | (codes[:, 1::2] << 4), "scale": scale.bfloat16(), "zero": zero,
            "table": table}


class _Pool:
    """The adapter pool that a serving program keeps, freed with the state."""

    def __init__(self, case, a, b, scales):
        import segmented_gathered_rank_amd as sgr
        self.sgr, m, page = sgr, _projections(case), case["page"]
        ranks = _ranks(case)
        pages = sum(ranks) * (case["h_in"] + case["h_out"]) // page * m
        self.h = sgr.lora_pool_create(torch.cuda.current_device(), sgr.LORA_BF16, page, pages, case["slots"], m,
                                      [case["h_in"]] * m, [case["h_out"]] * m, max(ranks))
        for s, r in enumerate(ranks):
            for p in range(m):
                sgr.lora_pool_load(self.h, s, p, r, a[p][s, :r].contiguous(), b[p][s, :r].contiguous(),
                                   float(scales[s]))
        torch.cuda.synchronize()

    def __del__(self):
        self.sgr.lora_pool_destroy(self.h)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n, h_in, h_out, slots = case["n"], case["h_in"], case["h_out"], case["slots"]
    st = {"case": case, "x": torch.randn(n, h_in, device=DEV, generator=g).bfloat16()}
    # runs of one adapter (prompts), or an adapter for each token; one run in nine has none
    run = case["run"]
    n_runs = -(-n // run)
    ids = torch.randint(0, slots, (n_runs,), device=DEV, generator=g, dtype=torch.int32)
    ids[8::9] = -1
    st["ids"] = ids.repeat_interleave(run)[:n].contiguous() if case["adapters"] else None
    st["w"] = [_weights(case, g) for _ in range(_projections(case))]
    ranks = _ranks(case)
    r_max = max(ranks)
    live = torch.tensor(ranks, device=DEV)[:, None, None] > torch.arange(r_max, device=DEV)[None, :, None]
    st["scales"] = [32.0 / r for r in ranks]
    st["a"] = [(torch.randn(slots, r_max, h_in, device=DEV, generator=g) * 0.02 * live).bfloat16() for _ in st["w"]]
    st["b"] = [(torch.randn(slots, r_max, h_out, device=DEV, generator=g) * 0.02 * live).bfloat16() for _ in st["w"]]
    if own:
        import segmented_gathered_rank_amd as sgr
        st["pool"] = _Pool(case, st["a"], st["b"], st["scales"])
        st["y"] = torch.empty(n, h_out, device=DEV, dtype=torch.bfloat16)
        st["ws"] = torch.empty(max(16, sgr.lora_fused_workspace_bytes(st["pool"].h, 0, len(st["w"]), n)), device=DEV,
                               dtype=torch.uint8)
        if case["group"]:
            st["w4"] = [sgr.lora_w4_bind(w["codes"], w["scale"], case["group"], zero=w["zero"], table=w["table"])
                        for w in st["w"]]
    return st


# ------------------------------------------------------------------ one pass
def _widened(case, w):
    """The base weights [h_out][h_in] in 32 bits."""
    if case["kind"] == "bf16":
        return w["w"].float()
    if case["kind"] == "fp8":
        return w["codes"].view(torch.float8_e4m3fn).float() * w["scale"][:, None]
    c = w["codes"]
    q = torch.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)
    q = w["table"].float()[q.int()] if w["table"] is not None else q.float()
    q = q.reshape(q.shape[0], -1, case["group"])
    if w["zero"] is not None:
        q = q - w["zero"].t().float()[:, :, None]
    elif w["table"] is None:
        q = q - 8.0
    return (q * w["scale"].t().float()[:, :, None]).reshape(c.shape[0], -1)


def _plain_linear(st, p):
    """x W + s (x A^T) B in 32 bits: the adapters of all slots side by side, each token's own kept by a mask."""
    case, x = st["case"], st["x"].float()
    y = x @ _widened(case, st["w"][p]).t()
    if st["ids"] is not None:
        a, b = st["a"][p].float(), st["b"][p].float()
        slots, r = a.shape[0], a.shape[1]
        t = x @ a.reshape(slots * r, -1).t()
        slot = torch.arange(slots, device=DEV).repeat_interleave(r)
        s = torch.tensor(st["scales"], device=DEV).repeat_interleave(r)
        t = torch.where(st["ids"][:, None] == slot[None, :], t * s, 0.0)
        y = y + t @ b.reshape(slots * r, -1)
    return y


def _plain_act(act, v):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))


def run(st):
    case = st["case"]
    if not own:
        y = _plain_linear(st, 0)
        if case["op"] == "glu":
            y = _plain_act(case["act"], y) * _plain_linear(st, 1)
        return y.bfloat16()
    import segmented_gathered_rank_amd as sgr
    pool, n, h_in, h_out = st["pool"].h, case["n"], case["h_in"], case["h_out"]
    act = {"silu": sgr.LORA_ACT_SILU, "gelu": sgr.LORA_ACT_GELU, "gelu_tanh": sgr.LORA_ACT_GELU_TANH}[case["act"]]
    w = st["w"]
    if case["op"] == "gemm":
        sgr.lora_fused_gemm_w4(pool, 0, st["x"], h_in, st["w4"][0], st["ids"], n, st["y"], h_out, st["ws"])
    elif case["kind"] == "bf16":
        sgr.lora_fused_glu(pool, 0, 1, st["x"], h_in, w[0]["w"], w[1]["w"], h_in, st["ids"], n, act, st["y"], h_out,
                           st["ws"])
    elif case["kind"] == "fp8":
        sgr.lora_fused_glu_fp8w(pool, 0, 1, st["x"], h_in, w[0]["codes"], w[1]["codes"], h_in, w[0]["scale"],
                                w[1]["scale"], st["ids"], n, act, st["y"], h_out, st["ws"])
    else:
        sgr.lora_fused_glu_w4(pool, 0, 1, st["x"], h_in, st["w4"][0], st["w4"][1], st["ids"], n, act, st["y"], h_out,
                              st["ws"])
    return st["y"]


def work(case):
    n, h_in, h_out, m = case["n"], case["h_in"], case["h_out"], _projections(case)
    per = {"bf16": 2.0, "fp8": 1.0}.get(case["kind"], 0.5)
    w = h_in * h_out * per
    if case["kind"] == "fp8":
        w += 4 * h_out
    if case["group"]:
        w += h_in // case["group"] * h_out * (3 if case["kind"] == "int4z" else 2)
    by, fl = 2 * n * (h_in + h_out) + m * w, 2 * n * h_in * h_out * m
    if case["adapters"]:
        ranks = _ranks(case)
        rank = sum(ranks) / len(ranks)
        distinct = case["slots"] * (1 - (1 - 1 / case["slots"]) ** -(-n // case["run"]))
        by += 4 * n + m * distinct * rank * (h_in + h_out) * 2
        fl += m * 2 * n * rank * (h_in + h_out)
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    x = st["x"].double()
    got = []
    for p, w in enumerate(st["w"]):
        if "w" in w:
            wt = w["w"].double().t()
        elif case["kind"] == "fp8":
            b = w["codes"].long()   # sign, 4 exponent bits (bias 7), 3 mantissa bits
            e, f = (b >> 3) & 15, (b & 7).double()
            mag = torch.where(e > 0, (1 + f / 8) * torch.exp2((e - 7).double()), f * 2.0 ** -9)
            wt = (torch.where(b > 127, -mag, mag) * w["scale"].double()[:, None]).t()
        else:
            k = torch.arange(case["h_in"], device=DEV)
            q = ((w["codes"].long()[:, k // 2] >> (4 * (k % 2))) & 15).t()   # [h_in][h_out]
            if w["table"] is not None:
                v = w["table"].double()[q]
            else:
                v = q.double() - (8.0 if w["zero"] is None else w["zero"].double()[k // case["group"]])
            wt = v * w["scale"].double()[k // case["group"]]
        y = x @ wt
        if st["ids"] is not None:
            for s, r in enumerate(_ranks(case)):
                i = (st["ids"] == s).nonzero()[:, 0]
                if i.numel():
                    t = x[i] @ st["a"][p][s, :r].double().t()
                    y[i] += st["scales"][s] * (t @ st["b"][p][s, :r].double())
        got.append(y)
    if case["op"] == "gemm":
        return got[0]
    gate, up = got
    if case["act"] == "silu":
        gate = gate * torch.sigmoid(gate)
    elif case["act"] == "gelu":
        gate = gate * torch.special.ndtr(gate)
    else:
        gate = gate * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))
    return gate * up
