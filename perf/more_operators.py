"""The measured passes of the operators around the plan that work on few bits or few numbers:
the experts' weights in 4 bits with group scales (packing, and the gated feed-forward
experts with rows in bf16 and in 8 bits), and the router, whose ids and weights the plan
takes (forward and backward).

`run` computes a pass in elementary torch operations where `own` is false and through the
library's entry points where it is true; `exact` computes it in 64 bits, from the
definitions alone.

Definitions.  4 bits: 32 neighbours along a matrix row share a power of two, the smallest (from
2^-126 on) that brings their largest magnitude to 6 or less, and each is one of 0, 0.5, 1,
1.5, 2, 3, 4, 6 with a sign, the nearest (ties to the even code), times it; the last block of a
row may be short.  8 bits: the same with e4m3, 448 and 2^-127.  A plan cuts the R*NvS buffer rows
into groups (each expert's rows on its home rank, each replica's in a prefetch slot,
fallback pieces); rows of no group are left as they were (zero here).  One expert has a gate
[I, H], an up [I, H] and a down [H, I] matrix.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
ROW_ALIGN = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------

def _named(name, c):
    return dict(c, name=name) if name else c


def _router(name, op, T, E, K, score="softmax", dtype="fp32", bias=False, groups=1, top_groups=1, normalize=True):
    return _named(name, dict(op=op, T=T, E=E, K=K, score=score, dtype=dtype, bias=bias, groups=groups,
                             top_groups=top_groups, normalize=normalize))


def _pack(name, n, H, I):
    return _named(name, dict(op="w4_pack", n=n, H=H, I=I))


def _ffn(name, op, R, E, K, S, slots, H, I, act="silu", skew=0.3, train=False):
    return _named(name, dict(op=op, R=R, E=E, K=K, S=S, slots=slots, H=H, I=I, act=act, skew=skew, train=train))


def listed():
    return [
        # a decode step's tokens: the launch is everything
        _router("router decode", "router", 8, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4),
        # prefill of many tokens to the most experts of the repository's workloads
        _router("router prefill", "router", 131072, 384, 8, score="sigmoid", bias=True),
        # training at the r8-e64-k6 workload's sizes, weights not normalised: every logit has a gradient
        _router("router backward", "router_bwd", 8192, 64, 6, normalize=False),
        # training at the widest setting, bf16 logits
        _router("router backward large", "router_bwd", 131072, 384, 8, score="sigmoid", dtype="bf16", bias=True),
        # a layer's experts packed once, as loaded
        _pack("pack", 16, 7168, 2048),
        # sizes that fill no block and no tile
        _pack("pack odd", 21, 1000, 680),
        # one decode step of a few sequences at the wide hidden size: most experts see one row or none
        _ffn("w4 decode", "ffn_w4", 8, 64, 8, 1, 3, 7168, 2048),
        # odd sizes, too few slots, the other activation, gate and up saved for a gradient of the rows
        _ffn("w4 odd", "ffn_w4", 3, 21, 3, 571, 1, 1000, 680, act="gelu", skew=1.0, train=True),
        # prefill with bf16 rows: hundreds of rows to an expert
        _ffn("w4 prefill", "ffn_w4", 8, 64, 6, 1024, 8, 2048, 1408),
        # a large decode batch with 8-bit rows: tens of rows to an expert
        _ffn("w4 q8 decode batch", "ffn_w4q8", 8, 64, 8, 64, 3, 7168, 2048),
        # 8-bit rows at sizes that fill no tile
        _ffn("w4 q8 odd", "ffn_w4q8", 3, 21, 3, 571, 1, 992, 672, act="gelu", skew=1.0),
        # prefill with 8-bit rows at the wide hidden size
        _ffn("w4 q8 prefill", "ffn_w4q8", 8, 32, 8, 512, 4, 7168, 2048),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["router", "router", "router_bwd", "w4_pack", "ffn_w4", "ffn_w4", "ffn_w4q8", "ffn_w4q8"])
    if op.startswith("router"):
        E = _spread(rng, 2, 1024)
        T = _spread(rng, 1, min(131072, 131072 * 384 // E))
        K = rng.randint(1, min(16, E))
        groups = rng.choice([g for g in (1, 1, 2, 3, 4, 7, 8, 16) if E % g == 0])
        top_groups = rng.choice([n for n in range(1, groups + 1) if n * (E // groups) >= K])
        return _router(None, op, T, E, K, score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["fp32", "bf16"]),
                       bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, normalize=rng.random() < 0.7)
    step = 32 if op == "ffn_w4q8" else 8
    if op == "w4_pack":
        H, I = _spread(rng, 64, 7168, step), _spread(rng, 32, 2048, step)
        return _pack(None, _spread(rng, 1, max(1, min(256, 16 * 7168 * 2048 // (H * I)))), H, I)
    while True:
        R = rng.choice([1, 2, 3, 4, 5, 8])
        E = R * _spread(rng, 1, 64 // R)
        K = rng.randint(1, min(8, E))
        H = _spread(rng, 64, 7168, step)
        I = _spread(rng, 32, 2048, step)
        S = _spread(rng, 1, 4096)
        slots = rng.choice([0, 1, 2, 4])
        A = R * S * K
        if A <= 32768 and A * H * I <= 16384 * 7168 * 2048 and E * H * I <= 32 * 7168 * 2048:
            break
    return _ffn(None, op, R, E, K, S, slots, H, I, act=rng.choice(["silu", "gelu"]), skew=round(rng.uniform(0.0, 1.0), 3),
                train=op == "ffn_w4" and rng.random() < 0.5)


def work(case):
    c = case
    if c["op"].startswith("router"):
        T, E, K = c["T"], c["E"], c["K"]
        size = 4 if c["dtype"] == "fp32" else 2
        if c["op"] == "router":              # logits in, ids and weights out
            return {"bytes": T * E * size + T * K * 8, "flops": 4 * T * E}
        # ids and the weights' gradient in, with the logits chosen or all of them; every logit's gradient out
        dense = c["score"] == "softmax" and not c["normalize"]
        return {"bytes": T * E * size * (2 if dense else 1) + T * K * (8 if dense else 8 + size), "flops": 4 * T * E}
    H, I = c["H"], c["I"]
    slab = 3 * H * I
    if c["op"] == "w4_pack":                 # bf16 in, 17 bytes of 32 out; those in and bf16 out
        return {"bytes": c["n"] * slab * (2 + 17 / 32) * 2, "flops": 4 * c["n"] * slab}
    A = c["R"] * c["S"] * c["K"]
    used = c["E"] * (1 - (1 - c["K"] / c["E"]) ** (c["R"] * c["S"]))     # experts with rows
    rows = A * H * (2 + 33 / 32) if c["op"] == "ffn_w4q8" else A * H * 4 + (A * I * 6 if c["train"] else 0)
    return {"bytes": used * slab * 17 / 32 + rows, "flops": 2.0 * A * slab}


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------

def _up16(n):
    return (n + ROW_ALIGN - 1) // ROW_ALIGN * ROW_ALIGN


def _groups(load, R, E, S, K, slots):
    """The plan rule on the experts' loads: rows of the whole buffer, and for each group
    (first row, rows, expert)."""
    e_loc, quota = E // R, S * K
    n_per_rank = _up16(quota + (e_loc + slots) * (ROW_ALIGN - 1))
    order = sorted(range(E), key=lambda e: (-load[e], e))
    home_load = [sum(load[r * e_loc:(r + 1) * e_loc]) for r in range(R)]
    excess = [max(0, v - quota) for v in home_load]
    need = [max(0, quota - v) for v in home_load]
    shed = [0] * E
    for e in order:
        shed[e] = min(load[e], excess[e // e_loc])
        excess[e // e_loc] -= shed[e]
    slot_rows = [[] for _ in range(R)]
    pieces, behind = [], [0] * R
    for e in order:
        left = shed[e]
        while left:
            r = next((r for r in range(R) if need[r] and len(slot_rows[r]) < slots), None)
            slot = -1
            if r is None:
                r = next(r for r in range(R) if need[r])
            else:
                slot = len(slot_rows[r])
            n = min(left, need[r])
            pieces.append((e, r, slot, n, behind[r]))
            if slot < 0:
                behind[r] += n
            else:
                slot_rows[r].append(n)
            need[r] -= n
            left -= n
    found, after, starts = [], [], []
    for r in range(R):
        at, slot_at = r * n_per_rank, []
        for e in range(r * e_loc, (r + 1) * e_loc):
            found.append((at, load[e] - shed[e], e))
            at += _up16(load[e] - shed[e])
        for s in range(slots):
            slot_at.append(at)
            at += _up16(slot_rows[r][s]) if s < len(slot_rows[r]) else 0
        starts.append(slot_at)
        after.append(at)
    for e, r, slot, n, pos in pieces:
        found.append((starts[r][slot] if slot >= 0 else after[r] + pos, n, e))
    return R * n_per_rank, [g for g in found if g[1]]


def _act(z, kind):
    if kind == "silu":
        return z * torch.sigmoid(z)
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def _normal(g, *shape, scale=1.0):
    t = torch.empty(*shape, dtype=torch.bfloat16, device=DEV)
    t.normal_(0.0, scale, generator=g)
    return t


def _blocks(v):
    """[rows, n] as [rows, blocks, 32], the last block filled up with zeros."""
    n = v.shape[1]
    if n % 32:
        v = torch.cat([v, v.new_zeros(v.shape[0], 32 - n % 32)], 1)
    return v.reshape(v.shape[0], -1, 32)


def _nibbles(w):
    """fp32 matrix rows in 4 bits: codes, one to a byte [rows, blocks, 32], and the powers of two's
    exponents [rows, blocks]."""
    b = _blocks(w)
    frac, exp = torch.frexp(b.abs().amax(2))               # largest = frac * 2^exp, 0.5 <= frac < 1
    exp = (exp - 3 + (frac > 0.75)).clamp_min(-126)
    m = torch.ldexp(b.abs(), -exp[:, :, None])
    # the border between two values goes to the one with the even code
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5))
    return (code | (b < 0).to(torch.uint8) << 3), exp


def _values(code, exp, n):
    """What codes and exponents stand for, fp32 [rows, n]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    return torch.ldexp(table[code.int()], exp[:, :, None]).reshape(code.shape[0], -1)[:, :n]


def _rows8(x):
    """bf16 rows as rows in 8 bits: e4m3 codes, a scale byte for 32, zeros up to a multiple of 16."""
    b = x.float().reshape(x.shape[0], -1, 32)
    frac, exp = torch.frexp(b.abs().amax(2))
    exp = (exp - 9 + (frac > 0.875)).clamp_min(-127)
    codes = torch.ldexp(b, -exp[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape[0], -1)
    row = torch.cat([codes, (exp + 127).to(torch.uint8)], 1)
    return torch.cat([row, row.new_zeros(row.shape[0], -row.shape[1] % 16)], 1).contiguous()


def _expand8(rows, n):
    """fp32 values of rows in 8 bits."""
    v = rows[:, :n].contiguous().view(torch.float8_e4m3fn).float().reshape(rows.shape[0], -1, 32)
    return torch.ldexp(v, rows[:, n:n + n // 32, None].int() - 127).reshape(rows.shape[0], n)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * seed + 29)
    if c["op"].startswith("router"):
        T, E, K = c["T"], c["E"], c["K"]
        c["logits"] = (1.5 * torch.randn(T, E, generator=g, device=DEV)).to(
            torch.float32 if c["dtype"] == "fp32" else torch.bfloat16)
        c["b"] = 0.05 * torch.randn(E, generator=g, device=DEV) if c["bias"] else None
        if c["op"] == "router_bwd":
            # the ids and the gradient of the weights that the rest of the layer hands back
            key = c["logits"].float() + (0 if c["b"] is None else c["b"])
            c["ids"] = torch.topk(key, K, dim=1)[1].to(torch.int32).contiguous()
            c["g_w"] = torch.randn(T, K, generator=g, device=DEV)
        return c
    H, I = c["H"], c["I"]
    if c["op"] == "w4_pack":
        c["w"] = _normal(g, c["n"], 3 * H * I, scale=1 / math.sqrt(H))
        return c
    R, E, K, S, slots = (c[k] for k in ("R", "E", "K", "S", "slots"))
    T = R * S
    z = torch.randn(E, generator=g, device=DEV)
    u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-12, 1 - 1e-7)
    top, ids = torch.topk(c["skew"] * z - torch.log(-torch.log(u)), K, dim=1)
    ids, weights = ids.to(torch.int32).contiguous(), torch.softmax(top, 1).contiguous()
    load = torch.bincount(ids.reshape(-1).long(), minlength=E).tolist()
    rows, c["groups"] = _groups(load, R, E, S, K, slots)
    c["rows"] = rows
    if own:
        import combine_top_id_amd as M
        c["plan"] = M.moonep_plan(ids, weights, R, E, K, S, slots)
        c["home_w4"] = torch.empty(E, M.moonep_w4_slab_bytes(H, I), dtype=torch.uint8, device=DEV)
    c["w4"] = []                                            # of each expert: codes two to a byte, and exponents
    for e in range(E):
        w = _normal(g, 3 * H * I, scale=1 / math.sqrt(H)).float()
        if own:                                             # packing rounds the same way
            M.moonep_w4_pack(w.to(torch.bfloat16)[None], H, I, out=c["home_w4"][e:e + 1])
            continue
        kept = []
        for m in (w[:2 * I * H].view(2 * I, H), w[2 * I * H:].view(H, I)):
            code, exp = _nibbles(m)
            kept.append((code[:, :, 0::2] | code[:, :, 1::2] << 4, exp.to(torch.int8)))
        c["w4"].append(kept)
    if own:
        c["slot_w4"] = M.moonep_prefetch_weight(c["plan"], c["home_w4"].view(torch.bfloat16)).view(torch.uint8)
    x = _normal(g, rows, H)
    c["recv"] = _rows8(x) if c["op"] == "ffn_w4q8" else x
    c["y"] = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    if c["op"] == "ffn_w4":
        c["h"] = torch.zeros(rows, I, dtype=torch.bfloat16, device=DEV)
        c["gu"] = torch.zeros(rows, 2 * I, dtype=torch.bfloat16, device=DEV) if c["train"] else None
    elif own:
        c["h"] = torch.zeros(rows, M.moonep_q8_row_bytes(I), dtype=torch.uint8, device=DEV)
    return c


# ----------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(c):
    import combine_top_id_amd as M
    op = c["op"]
    if op == "router":
        return M.moonep_router(c["logits"], c["K"], bias=c["b"], score=c["score"], groups=c["groups"],
                               top_groups=c["top_groups"], normalize=c["normalize"], scale=2.5)
    if op == "router_bwd":
        return M.moonep_router_bwd(c["logits"], c["ids"], c["g_w"], score=c["score"], normalize=c["normalize"], scale=2.5)
    if op == "w4_pack":
        return M.moonep_w4_unpack(M.moonep_w4_pack(c["w"], c["H"], c["I"]), c["H"], c["I"])
    if op == "ffn_w4":
        y, h, gu = M.moonep_expert_ffn_w4(c["plan"], c["recv"], c["home_w4"], c["slot_w4"], c["I"], act=c["act"], h=c["h"],
                                          gu=c["gu"], y=c["y"])
        return (y, h, gu) if c["train"] else y
    return M.moonep_expert_ffn_w4q8(c["plan"], c["recv"], c["home_w4"], c["slot_w4"], c["H"], c["I"], act=c["act"],
                                    h=c["h"], y=c["y"])[0]


def _scores(l, kind):
    return torch.softmax(l, 1) if kind == "softmax" else torch.sigmoid(l)


def _matrix(kept, n):
    """One matrix's fp32 values from its codes and exponents."""
    two, exp = kept
    code = torch.stack([two & 15, two >> 4], 3).reshape(two.shape[0], two.shape[1], 32)
    return _values(code, exp.int(), n)


def _run_plain(c):
    op = c["op"]
    if op == "router":
        T, E, K, n = c["T"], c["E"], c["K"], c["groups"]
        # scores that differ little are told apart in 64 bits
        key = _scores(c["logits"].double(), c["score"])
        if c["b"] is not None:
            key = key + c["b"].double()
        if n > 1:
            two = torch.sort(key.view(T, n, E // n), 2, descending=True)[0][:, :, :2].sum(2)
            best = torch.sort(two, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
            live = torch.zeros(T, n, dtype=torch.bool, device=DEV).scatter_(1, best, True)
            key = torch.where(live[:, :, None], key.view(T, n, E // n), -math.inf).view(T, E)
        ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :K]
        w = torch.gather(_scores(c["logits"].float(), c["score"]), 1, ids)
        if c["normalize"]:
            w = w / w.sum(1, keepdim=True)
        return ids.to(torch.int32), 2.5 * w
    if op == "router_bwd":
        l, ids, g = c["logits"].float(), c["ids"].long(), 2.5 * c["g_w"]
        s = _scores(l, c["score"])
        p = torch.gather(s, 1, ids)
        if c["normalize"]:                  # of the scores: the gradient through the division
            g = (g - (g * p).sum(1, keepdim=True) / p.sum(1, keepdim=True)) / p.sum(1, keepdim=True)
        g = torch.zeros_like(l).scatter_(1, ids, g)
        g = s * (g - (g * s).sum(1, keepdim=True)) if c["score"] == "softmax" else g * s * (1 - s)
        return g.to(c["logits"].dtype)
    H, I = c["H"], c["I"]
    if op == "w4_pack":
        out = torch.empty_like(c["w"])
        for w, o in zip(c["w"], out):
            o[:2 * I * H] = _values(*_nibbles(w[:2 * I * H].float().view(2 * I, H)), H).reshape(-1)
            o[2 * I * H:] = _values(*_nibbles(w[2 * I * H:].float().view(H, I)), I).reshape(-1)
        return out
    y = torch.zeros_like(c["y"])
    save = c["train"]
    hs = torch.zeros_like(c["h"]) if save else None
    gus = torch.zeros_like(c["gu"]) if save else None
    for r0, n, e in c["groups"]:
        gate_up, down = _matrix(c["w4"][e][0], H), _matrix(c["w4"][e][1], I)
        x = c["recv"][r0:r0 + n]
        x = _expand8(x, H) if op == "ffn_w4q8" else x.float()
        gu = x @ gate_up.T
        h = _act(gu[:, :I], c["act"]) * gu[:, I:]
        if save:
            hs[r0:r0 + n], gus[r0:r0 + n] = h.to(torch.bfloat16), gu.to(torch.bfloat16)
        if op == "ffn_w4q8":                # the second product takes rows in 8 bits too
            b = h.reshape(n, -1, 32)
            frac, exp = torch.frexp(b.abs().amax(2, keepdim=True))
            exp = (exp - 9 + (frac > 0.875)).clamp_min(-127)
            h = torch.ldexp(torch.ldexp(b, -exp).to(torch.float8_e4m3fn).float(), exp).reshape(n, I)
        y[r0:r0 + n] = (h @ down.T).to(torch.bfloat16)
    return (y, hs, gus) if save else y


# ----------------------------------------------------------------------------------------
# the same in 64 bits
# ----------------------------------------------------------------------------------------

def _exact_scores(l, kind):
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.max(1, keepdim=True)[0])
    return e / e.sum(1, keepdim=True)


def _take(key, n):
    """Columns of the n largest of each row, the lowest where they are equal."""
    key, cols, got = key.clone(), torch.arange(key.shape[1], device=DEV), []
    for _ in range(n):
        top = key.max(1, keepdim=True)[0]
        i = torch.where(key == top, cols, key.shape[1]).min(1, keepdim=True)[0]
        key.scatter_(1, i, -math.inf)
        got.append(i)
    return torch.cat(got, 1)


def _exact_router(c, l, ids, g):
    s = _exact_scores(l.double(), c["score"])
    if c["op"] == "router":
        key = s if c["b"] is None else s + c["b"].double()
        if c["groups"] > 1:
            k = key.view(len(l), c["groups"], -1)
            best = k.max(2)[0]
            if k.shape[2] > 1:
                rest = k.reshape(-1, k.shape[2])
                rest = rest.scatter(1, _take(rest, 1), -math.inf)
                best = best + rest.max(1)[0].view_as(best)
            keep = torch.full_like(best, -math.inf).scatter_(1, _take(best, c["top_groups"]), 0.0)
            key = (k + keep[:, :, None]).reshape(key.shape)
        ids = _take(key, c["K"])
        w = torch.gather(s, 1, ids)
        return ids.to(torch.int32), 2.5 * (w / w.sum(1, keepdim=True) if c["normalize"] else w)
    sel = torch.gather(s, 1, ids.long())
    g = 2.5 * g.double()
    if c["normalize"]:
        p = sel / sel.sum(1, keepdim=True)
        d = p * (g - (g * p).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1 - sel)
        return torch.zeros_like(s).scatter_(1, ids.long(), d)
    if c["score"] == "sigmoid":
        return torch.zeros_like(s).scatter_(1, ids.long(), g * sel * (1 - sel))
    out = -s * (g * sel).sum(1, keepdim=True)
    return out.scatter_add_(1, ids.long(), g * sel)


def _exact_act(z, kind):
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
    return z * (1 - 1 / (1 + torch.exp(u)))


def _exact_round(v, most, bits, least, floor):
    """Blocks [.., 32] on the grid of an 8- or 4-bit form: `most` its largest value, `bits` of fraction
    from the power of two `least` on, scales from `floor` on."""
    top = v.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-300) / most)).clamp_min(floor))
    m = v.abs() / scale
    grid = torch.exp2(torch.floor(torch.log2(m.clamp_min(2.0 ** least))) - bits)
    return torch.sign(v) * torch.round(m / grid) * grid * scale


def _exact_w4(w, rows, n):
    """A bf16 matrix as its 4-bit values, 64 bits."""
    w = w.double().view(rows, n)
    w = torch.nn.functional.pad(w, (0, -n % 32)).view(rows, -1, 32)
    return _exact_round(w, 6.0, 1, 0, -126).reshape(rows, -1)[:, :n]


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op.startswith("router"):
        parts = []
        for at in range(0, c["T"], 16384):
            part = slice(at, at + 16384)
            parts.append(_exact_router(c, c["logits"][part], *((c["ids"][part], c["g_w"][part]) if op == "router_bwd" else (None, None))))
        if op == "router":
            return tuple(torch.cat(p) for p in zip(*parts))
        return torch.cat(parts)
    H, I = c["H"], c["I"]
    if op == "w4_pack":
        out = torch.empty(c["n"], 3 * H * I, device=DEV)          # values of few bits: fp32 holds them
        for w, o in zip(c["w"], out):
            o[:2 * I * H] = _exact_w4(w[:2 * I * H], 2 * I, H).reshape(-1)
            o[2 * I * H:] = _exact_w4(w[2 * I * H:], H, I).reshape(-1)
        return out
    # the weights again, from the same random numbers
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * seed + 29)
    torch.randn(c["E"], generator=g, device=DEV)
    torch.rand(c["R"] * c["S"], c["E"], generator=g, device=DEV)
    per = {}
    for group in c["groups"]:
        per.setdefault(group[2], []).append(group)
    rows = c["rows"]
    wide = torch.zeros(rows, H, dtype=torch.float64, device=DEV)
    mid = torch.zeros(rows, I, dtype=torch.float64, device=DEV) if c["train"] else None
    both = torch.zeros(rows, 2 * I, dtype=torch.float64, device=DEV) if c["train"] else None
    for e in range(c["E"]):
        w = _normal(g, 3 * H * I, scale=1 / math.sqrt(H))
        if e not in per:
            continue
        gate, up = _exact_w4(w[:I * H], I, H), _exact_w4(w[I * H:2 * I * H], I, H)
        down = _exact_w4(w[2 * I * H:], H, I)
        for r0, n, _ in per[e]:
            at = slice(r0, r0 + n)
            if op == "ffn_w4q8":
                scale = torch.exp2(c["recv"][at, H:H + H // 32].double() - 127)
                x = c["recv"][at, :H].contiguous().view(torch.float8_e4m3fn).double() * scale.repeat_interleave(32, 1)
            else:
                x = c["recv"][at].double()
            z, v = x @ gate.T, x @ up.T
            h = _exact_act(z, c["act"]) * v
            if c["train"]:
                mid[at], both[at, :I], both[at, I:] = h, z, v
            if op == "ffn_w4q8":
                h = _exact_round(h.view(n, -1, 32), 448.0, 3, -6, -127).reshape(n, I)
            wide[at] = h @ down.T
    return (wide, mid, both) if c["train"] else wide
