"""The measured cases of the experts' matrix products in 16 and 8 bits.

Five operators of the routed-expert layer, each over rows bucketed by expert
(rows offsets[e] to offsets[e+1] belong to expert e):

  mm       y[r, n]     = sum_k x[r, k] w[e, n, k]            bf16 or fp16
  dgrad    dx[r, k]    = sum_n dy[r, n] w[e, n, k]           its gradient by x
  wgrad    dw[e, n, k] = sum_{r of e} dy[r, n] x[r, k]       its gradient by w, 16 bits or fp32
  swiglu8  h[r, f]     = silu(g) u, g and u 8-bit integer products of token
           row_slot[r] // top_k with gate and up, a scale for each token and each channel
  down8    y[r, n]     = topk_w[slot] * the same product of h[r] with down

8 bits: a row is quantised to q = rint(127 x / max|x|) with the scale
max|x| / 127; weights are int8 [E, out, in] with fp32 scales [E, out].
"""
import math

import numpy as np
import torch

own = False     # the tools set it: False, run() in plain torch; True, run() through the framework

F16 = {"bf16": torch.bfloat16, "fp16": torch.float16}
OUT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    c = []
    # 16-bit products.  One decode step of 8 tokens over 352 unquantised experts: the weight stream.
    c.append(dict(name="mm_decode_bf16", op="mm", E=352, T=8, k=8, K=4096, N=1536, dtype="bf16", load="even"))
    # the small layer at a 16-token step: launch latency
    c.append(dict(name="mm_small_fp16", op="mm", E=32, T=16, k=8, K=1024, N=256, dtype="fp16", load="even"))
    # a training step's rows on one of eight ranks (44 of 352 experts), uneven load
    c.append(dict(name="mm_train_bf16", op="mm", E=44, T=8192, k=8, K=4096, N=1536, dtype="bf16", load="zipf"))
    # gradient by the input: a small ragged batch, widths that fill no tile
    c.append(dict(name="dgrad_small_fp16", op="dgrad", E=32, T=37, k=8, K=1000, N=264, dtype="fp16", load="even"))
    # gradient by the input at the training step's rows
    c.append(dict(name="dgrad_train_bf16", op="dgrad", E=44, T=8192, k=8, K=4096, N=1536, dtype="bf16", load="zipf"))
    # gradient by the weights of every expert from a short batch (about 47 rows an expert): the write stream
    c.append(dict(name="wgrad_wide_bf16", op="wgrad", E=352, T=2047, k=8, K=4096, N=1536, dtype="bf16", out="bf16",
                  load="even"))
    # gradient by the weights at the training step's rows, kept in fp32 for the optimiser
    c.append(dict(name="wgrad_train_f32", op="wgrad", E=44, T=8192, k=8, K=4096, N=1536, dtype="bf16", out="f32",
                  load="zipf"))
    # 8-bit experts.  Decode steps: 8 tokens through gate and up, one token through down.
    c.append(dict(name="swiglu8_decode", op="swiglu8", E=352, T=8, k=8, K=4096, N=1536, load="even"))
    c.append(dict(name="down8_one_token", op="down8", E=352, T=1, k=8, K=1536, N=4096, load="even"))
    # a prompt of 2048 tokens, even load; a long prompt whose experts' load follows Zipf
    c.append(dict(name="down8_prompt", op="down8", E=352, T=2048, k=8, K=1536, N=4096, load="even"))
    c.append(dict(name="swiglu8_long", op="swiglu8", E=352, T=8192, k=8, K=4096, N=1536, load="zipf"))
    # one expert that owns every token (the shared expert in 8 bits), an odd batch
    c.append(dict(name="swiglu8_shared", op="swiglu8", E=1, T=61, k=1, K=4096, N=1536, load="even"))
    return c


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["mm", "dgrad", "wgrad", "swiglu8", "down8"])
        c = dict(op=op, E=_log_int(rng, 1, 352), T=_log_int(rng, 1, 8192), load=rng.choice(["even", "zipf"]))
        c["k"] = rng.randint(1, min(8, c["E"]))
        if op in ("mm", "dgrad", "wgrad"):
            c["K"] = 8 * _log_int(rng, 8, 512)
            c["N"] = 8 * _log_int(rng, 8, 192)
            c["dtype"] = rng.choice(["bf16", "fp16"])
            if op == "wgrad":
                c["out"] = rng.choice([c["dtype"], "f32"])
        else:
            wide, narrow = 128 * _log_int(rng, 2, 32), 128 * _log_int(rng, 1, 12)
            c["K"], c["N"] = (wide, narrow) if op == "swiglu8" else (narrow, wide)
        w = work(c)
        if w["bytes"] <= 7.0e9 and w["flops"] <= 1.7e12:      # no more than the largest listed case
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _load(case):
    """Expected share of the tokens' choices by expert."""
    E = case["E"]
    p = np.ones(E) if case["load"] == "even" else 1.0 / np.arange(1, E + 1) ** 1.1
    return p / p.sum()


def _inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    E, T, k, K, N, op = case["E"], case["T"], case["k"], case["K"], case["N"], case["op"]
    R = T * k
    # routing: k different experts for each token (Gumbel top-k over the load), rows stably bucketed by expert
    logp = torch.from_numpy(np.log(_load(case))).to(dev, torch.float32)
    logp = logp[torch.randperm(E, generator=g, device=dev)]
    u = torch.rand(T, E, generator=g, device=dev).clamp_(1e-9, 1 - 1e-7)
    ids = torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices
    flat = ids.reshape(-1)
    slots = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    off[1:] = torch.cumsum(counts, 0)
    d = {"case": case, "offsets": off.to(torch.int32), "row_slot": slots.to(torch.int32), "bounds": off.tolist()}

    def normal(*shape, dtype, std):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(std)

    def int8_bank(n_out, n_in):
        q = torch.empty(E, n_out, n_in, dtype=torch.int8, device=dev)
        step = max(1, (1 << 28) // (n_out * n_in))
        for e in range(0, E, step):                      # gaussian weights: a row's largest is near 3.7 sigma
            w = torch.randn(min(step, E - e), n_out, n_in, generator=g, device=dev, dtype=torch.bfloat16)
            q[e:e + step] = w.mul_(34.0).round_().clamp_(-127, 127).to(torch.int8)
        s = (0.02 / 34.0) * (0.8 + 0.4 * torch.rand(E, n_out, generator=g, device=dev))
        return q, s

    if op in ("mm", "dgrad", "wgrad"):
        dt = F16[case["dtype"]]
        if op != "wgrad":
            d["w"] = normal(E, N, K, dtype=dt, std=0.02)
        if op != "dgrad":
            d["x"] = normal(R, K, dtype=dt, std=1.0)
        if op != "mm":
            d["dy"] = normal(R, N, dtype=dt, std=0.1)
    elif op == "swiglu8":
        x = normal(T, K, dtype=torch.float32, std=1.0)
        x[:, torch.randint(0, K, (max(1, K // 512),), generator=g, device=dev)] *= 8.0     # outlier channels
        d["x"] = x.to(torch.bfloat16)
        d["gate"], d["up"] = int8_bank(N, K), int8_bank(N, K)
    else:
        a, b = normal(R, K, dtype=torch.float32, std=1.3), normal(R, K, dtype=torch.float32, std=1.3)
        d["x"] = (a * torch.sigmoid(a) * b).to(torch.bfloat16)          # what silu(g) u leaves
        d["down"] = int8_bank(N, K)
        w = torch.rand(T, k, generator=g, device=dev) + 0.1
        d["topk_w"] = (w / w.sum(1, keepdim=True)).reshape(-1).contiguous()
    return d


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from weight_only_bit_route_b200 import moe
        st["moe"] = moe
        if case["op"] in ("mm", "dgrad", "wgrad"):
            st["ws"] = moe.control_block()
        else:
            H, F = (case["K"], case["N"]) if case["op"] == "swiglu8" else (case["N"], case["K"])
            st["ws"] = moe.workspace(case["T"], H, case["E"], F, case["k"])
            for b in ("gate", "up", "down"):
                if b in st:
                    st[b] = moe.Bank(moe.FMT_INT8, *st[b])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _experts(bounds):
    return [(e, a, b) for e, (a, b) in enumerate(zip(bounds, bounds[1:])) if b > a]


def _quantised(x):
    """Rows as whole numbers in [-127, 127] (held in fp32) and the scale of each row."""
    x = x.float()
    amax = x.abs().amax(dim=1, keepdim=True)
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    return torch.round(x * 127.0 / safe), (amax / torch.full_like(amax, 127.0))


def _plain(st):
    c = st["case"]
    op, rows = c["op"], c["T"] * c["k"]
    if op == "mm":
        y = torch.empty(rows, c["N"], dtype=F16[c["dtype"]], device="cuda")
        for e, a, b in _experts(st["bounds"]):
            y[a:b] = torch.matmul(st["x"][a:b].float(), st["w"][e].float().t())
        return y
    if op == "dgrad":
        dx = torch.empty(rows, c["K"], dtype=F16[c["dtype"]], device="cuda")
        for e, a, b in _experts(st["bounds"]):
            dx[a:b] = torch.matmul(st["dy"][a:b].float(), st["w"][e].float())
        return dx
    if op == "wgrad":
        dw = torch.zeros(c["E"], c["N"], c["K"], dtype=OUT[c["out"]], device="cuda")
        for e, a, b in _experts(st["bounds"]):
            dw[e] = torch.matmul(st["dy"][a:b].float().t(), st["x"][a:b].float())
        return dw
    q, s = _quantised(st["x"])
    slot = st["row_slot"].long()
    y = torch.empty(rows, c["N"], dtype=torch.bfloat16, device="cuda")
    for e, a, b in _experts(st["bounds"]):
        if op == "swiglu8":
            t = slot[a:b] // c["k"]
            gate = torch.matmul(q[t], st["gate"][0][e].float().t()) * (s[t] * st["gate"][1][e])
            up = torch.matmul(q[t], st["up"][0][e].float().t()) * (s[t] * st["up"][1][e])
            y[a:b] = gate / (1.0 + torch.exp(-gate)) * up
        else:
            p = torch.matmul(q[a:b], st["down"][0][e].float().t()) * (s[a:b] * st["down"][1][e])
            y[a:b] = p * st["topk_w"][slot[a:b]].unsqueeze(1)
    return y


def run(st):
    if not own:
        return _plain(st)
    moe, c = st["moe"], st["case"]
    op = c["op"]
    if op == "mm":
        return moe.grouped_mm(st["x"], st["w"], st["offsets"], st["ws"])
    if op == "dgrad":
        return moe.grouped_mm_dgrad(st["dy"], st["w"], st["offsets"], st["ws"])
    if op == "wgrad":
        return moe.grouped_mm_wgrad(st["dy"], st["x"], st["offsets"], st["ws"], out_dtype=OUT[c["out"]])
    if op == "swiglu8":
        return moe.grouped_swiglu(st["x"], st["offsets"], st["row_slot"], c["k"], st["gate"], st["up"],
                                  c["T"] * c["k"], st["ws"])
    return moe.grouped_down(st["x"], st["offsets"], st["row_slot"], st["topk_w"], st["down"], st["ws"])


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the operators in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    E, T, k, K, N, op = case["E"], case["T"], case["k"], case["K"], case["N"], case["op"]
    R = T * k
    # experts that some token chose: each token takes k different ones
    touched = float(np.minimum(1.0, 1.0 - (1.0 - np.minimum(1.0, k * _load(case))) ** T).sum())
    if op in ("mm", "dgrad"):
        return {"bytes": 2.0 * (touched * N * K + R * (N + K)) + 4 * (E + 1), "flops": 2.0 * R * N * K}
    if op == "wgrad":
        size = 4.0 if case["out"] == "f32" else 2.0
        return {"bytes": 2.0 * R * (N + K) + size * E * N * K + 4 * (E + 1), "flops": 2.0 * R * N * K}
    banks, xrows = (2, T) if op == "swiglu8" else (1, R)
    small = 4.0 * (E + 1 + R) + (4.0 * R if op == "down8" else 0.0)
    return {"bytes": banks * touched * (N * K + 4.0 * N) + 2.0 * (xrows * K + R * N) + small,
            "flops": 2.0 * banks * R * N * K}


def exact(case, seed):
    d = _inputs(case, seed)
    op, E, k = case["op"], case["E"], case["k"]
    f64 = torch.float64
    spans = [range(d["bounds"][e], d["bounds"][e + 1]) for e in range(E)]
    if op == "wgrad":
        res = torch.zeros(E, case["N"], case["K"], dtype=f64, device="cuda")
    else:
        res = torch.zeros(case["T"] * k, case["K"] if op == "dgrad" else case["N"], dtype=f64, device="cuda")
    for e, span in enumerate(spans):
        if len(span) == 0:
            continue
        i = slice(span.start, span.stop)
        if op == "mm":
            res[i] = d["x"][i].to(f64) @ d["w"][e].to(f64).mT
        elif op == "dgrad":
            res[i] = d["dy"][i].to(f64) @ d["w"][e].to(f64)
        elif op == "wgrad":
            res[e] = d["dy"][i].to(f64).mT @ d["x"][i].to(f64)
        else:
            slots = d["row_slot"][i].long()
            src = d["x"][slots.div(k, rounding_mode="floor")] if op == "swiglu8" else d["x"][i]
            v = src.to(f64)
            top = v.abs().max(dim=1, keepdim=True).values
            codes = torch.where(top > 0, torch.round(v * 127.0 / torch.where(top > 0, top, 1.0)), 0.0)

            def product(bank):
                return (codes @ bank[0][e].to(f64).mT) * (top / 127.0) * bank[1][e].to(f64)

            if op == "swiglu8":
                g = product(d["gate"])
                res[i] = g * torch.sigmoid(g) * product(d["up"])
            else:
                res[i] = product(d["down"]) * d["topk_w"].to(f64)[slots].unsqueeze(1)
    return res
