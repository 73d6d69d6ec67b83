"""Cases of the mixture-of-experts operators: routing, grouping and combining,
FP8 quantisation, and the grouped FP8 products.

Sizes are those of the framework's workloads: 512 experts of 1536 x 4096
with hidden size 4096, a shared expert of 6144 x 4096, experts of
2048 x 8704 with hidden size 8704, top-7 routing.
"""

import functools

import numpy as np
import torch

own = False

TOPK = 7
BLOCK = 128
F8 = torch.float8_e4m3fn


@functools.lru_cache(maxsize=1)
def _lib():
    import newton_schulz_03_gb300 as ns
    return ns, ns.Handle()


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One generated token's routing over 512 experts (serving latency).
        dict(name="route one token", op="route", tokens=1, experts=512, k=TOPK, score="sigmoid", bias=True, groups=1,
             top_groups=1, group_top=1, renorm=True, dtype="float32", backward=False),
        # A training micro-batch: softmax routing with its backward pass.
        dict(name="route training batch", op="route", tokens=16384, experts=512, k=TOPK, score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=False, dtype="float32", backward=True),
        # A large batch with balance bias and expert groups, BF16 logits.
        dict(name="route groups", op="route", tokens=65531, experts=512, k=TOPK, score="sigmoid", bias=True, groups=16,
             top_groups=4, group_top=2, renorm=True, dtype="bfloat16", backward=True),
        # A small serving batch: group the slots, add up the experts' rows.
        dict(name="combine serving", op="combine", tokens=37, hidden=4096, experts=512, k=TOPK, backward=False),
        # A training micro-batch of odd length, both directions.
        dict(name="combine training", op="combine", tokens=8191, hidden=4096, experts=512, k=TOPK, backward=True),
        # Tokens quantised and sent to their experts' rows.
        dict(name="quantise tokens", op="rows", tokens=8192, hidden=4096, experts=512, k=TOPK),
        # FP32 master weights of 48 experts, for both directions of the product.
        dict(name="quantise weights", op="blocks", experts=48, rows=2048, cols=8704, dtype="float32"),
        # The gathered tokens along each expert's rows, for the weight gradient.
        dict(name="quantise columns", op="cols", tokens=8191, hidden=4096, experts=512, k=TOPK),
        # One generated token through its 7 experts out of 512.
        dict(name="experts one token", op="product", rows=TOPK, experts=512, active=TOPK, out=1536, hidden=4096),
        # A training micro-batch over all 512 experts, uneven.
        dict(name="experts training", op="product", rows=57344, experts=512, active=512, out=1536, hidden=4096),
        # The shared expert: a dense product with an odd number of tokens.
        dict(name="shared expert", op="product", rows=16381, experts=1, active=1, out=6144, hidden=4096),
        # Weight gradients of 64 large experts, some of them without tokens.
        dict(name="weight gradient", op="wgrad", rows=9000, experts=64, active=61, out=2048, hidden=8704),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "combine", "rows", "blocks", "cols", "product", "product", "wgrad"])
    if op == "route":
        experts = rng.choice([8, 64, 96, 256, 512, 1000])
        score = rng.choice(["sigmoid", "softmax"])
        groups = rng.choice([1, 4, 8])
        bias = score == "sigmoid" and rng.random() < 0.6
        return dict(op=op, tokens=_log(rng, 1, 65536), experts=experts, k=min(rng.choice([1, 2, 4, TOPK, 8]), experts // groups),
                    score=score, bias=bias, groups=groups, top_groups=max(1, groups // 2),
                    group_top=2 if score == "sigmoid" and groups > 1 and rng.random() < 0.5 else 1,
                    renorm=rng.random() < 0.5, dtype=rng.choice(["float32", "bfloat16"]), backward=rng.random() < 0.7)
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 8192), hidden=16 * _log(rng, 16, 256), experts=rng.choice([8, 64, 512]), k=rng.choice([1, 2, 4, TOPK]),
                    backward=rng.random() < 0.6)
    if op in ("rows", "cols"):
        return dict(op=op, tokens=_log(rng, 1, 8192), hidden=16 * _log(rng, 16, 256), experts=rng.choice([8, 64, 512]), k=rng.choice([1, 2, 4, TOPK]))
    if op == "blocks":
        return dict(op=op, experts=_log(rng, 1, 48), rows=16 * _log(rng, 16, 128), cols=16 * _log(rng, 16, 544),
                    dtype=rng.choice(["float32", "bfloat16"]))
    if op == "product":
        experts = rng.choice([1, 8, 64, 256])
        return dict(op=op, rows=_log(rng, 1, 32768), experts=experts, active=max(1, int(experts * (0.3 + 0.7 * rng.random()))),
                    out=16 * _log(rng, 16, 256), hidden=16 * _log(rng, 16, 256))
    experts = rng.choice([1, 8, 32])
    return dict(op=op, rows=_log(rng, 1, 16384), experts=experts, active=max(1, int(experts * (0.3 + 0.7 * rng.random()))),
                out=16 * _log(rng, 16, 256), hidden=16 * _log(rng, 16, 256))


# ------------------------------------------------------------------ inputs
def _up(a, b):
    return -(-a // b)


def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _routing(tokens, experts, k, g):
    """Distinct experts of each token, some experts more popular than others."""
    gum = -torch.log(-torch.log(torch.rand(tokens, experts, generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    gum += torch.randn(experts, generator=g, device="cuda") * 0.4
    return torch.topk(gum, k, dim=1).indices.int().contiguous()


def _group(ids, experts):
    flat = ids.reshape(-1).long()
    slots = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(slots)
    pos[slots] = torch.arange(slots.numel(), device="cuda")
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.bincount(flat, minlength=experts).cumsum(0)
    return offsets.int(), slots.int(), pos.int().reshape(ids.shape)


def _counts(case, seed):
    """Rows of each expert: `active` of them share the rows unevenly."""
    r = np.random.default_rng(seed)
    share = np.zeros(case["experts"])
    share[r.permutation(case["experts"])[:case["active"]]] = np.exp(r.laplace(0.0, 0.3, case["active"]))
    if case["rows"] == case["active"]:
        return (share > 0).astype(np.int64)
    return r.multinomial(case["rows"], share / share.sum()).astype(np.int64)


def _fp8(shape, g, std=100.0):
    out = torch.empty(shape, dtype=F8, device="cuda")
    flat = out.view(torch.uint8).view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        v = torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std).clamp_(-448, 448)
        flat[i:i + n] = v.to(F8).view(torch.uint8)
    return out


def _scales(shape, g, lo, hi):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8)


def _padded(counts, unit):
    """Of each group: its rows (or blocks) in a padded grid, the number of all standing for none."""
    n = -(-counts // unit)
    start = np.concatenate([[0], np.cumsum(n)])
    most = max(1, int(n.max()))
    at = start[:-1, None] + np.arange(most)[None]
    inside = np.arange(most)[None] < n[:, None]
    return n, start, np.where(inside, at, start[-1]), most


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        dt = getattr(torch, case["dtype"])
        st["logits"] = (torch.randn(T, E, generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda") * 0.5).to(dt)
        # A balance bias moves in steps of 0.001 as training goes on.
        st["bias"] = torch.randint(-60, 61, (E,), generator=g, device="cuda").float() * 0.001 if case["bias"] else None
        st["grad"] = torch.randn(T, k, generator=g, device="cuda")
        st["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty(T, k, device="cuda")
        st["grad_logits"] = torch.empty(T, E, dtype=dt, device="cuda")
    elif op in ("combine", "rows", "cols"):
        T, d, E, k = case["tokens"], case["hidden"], case["experts"], case["k"]
        st["ids"] = _routing(T, E, k, g)
        st["offsets"], st["slots"], st["pos"] = _group(st["ids"], E)
        R = T * k
        if op == "combine":
            st["y"] = torch.randn(R, d, generator=g, device="cuda", dtype=torch.bfloat16)
            st["weights"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
            st["grad"] = torch.randn(T, d, generator=g, device="cuda", dtype=torch.bfloat16)
            st["out"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
            st["grad_y"] = torch.empty(R, d, dtype=torch.bfloat16, device="cuda")
            st["grad_w"] = torch.empty(T, k, device="cuda")
            st["plan"] = [torch.empty_like(st[n]) for n in ("offsets", "slots", "pos")]
        else:
            # Activations with a few large channels.
            st["x"] = (torch.randn(T, d, generator=g, device="cuda") * torch.exp(torch.randn(d, generator=g, device="cuda"))).bfloat16()
        if op == "rows":
            st["q"] = torch.empty(R, d, dtype=F8, device="cuda")
            st["s"] = torch.empty(R, _up(d, BLOCK), dtype=torch.uint8, device="cuda")
        elif op == "cols":
            counts = (st["offsets"][1:] - st["offsets"][:-1]).cpu().numpy()
            n, start, at, most = _padded(counts, BLOCK)
            # The row that each padded place holds (R: none); the buffers hold
            # the padding of any routing, and stay zero past this one's.
            P = (R + (BLOCK - 1) * min(E, R)) // BLOCK * BLOCK
            place = np.full(P, R, dtype=np.int64)
            begin = np.concatenate([[0], np.cumsum(counts)])
            for e in range(E):
                place[start[e] * BLOCK:start[e] * BLOCK + counts[e]] = np.arange(begin[e], begin[e + 1])
            st["place"] = torch.from_numpy(place).cuda()
            st["used"] = torch.arange(P // BLOCK, device="cuda") < int(start[-1])
            st["q"] = torch.zeros(d, P, dtype=torch.uint8, device="cuda").view(F8)
            st["s"] = torch.zeros(P // BLOCK, d, dtype=torch.uint8, device="cuda")
    elif op == "blocks":
        E, N, K = case["experts"], case["rows"], case["cols"]
        st["w"] = (torch.randn(E, N, K, generator=g, device="cuda") * 0.02).to(getattr(torch, case["dtype"]))
        st["q"] = torch.empty(E, N, K, dtype=F8, device="cuda")
        st["s"] = torch.empty(E, _up(N, BLOCK), _up(K, BLOCK), dtype=torch.uint8, device="cuda")
        st["qt"] = torch.empty(E, K, N, dtype=F8, device="cuda")
        st["st"] = torch.empty(E, _up(K, BLOCK), _up(N, BLOCK), dtype=torch.uint8, device="cuda")
    else:
        E, N, K, R = case["experts"], case["out"], case["hidden"], case["rows"]
        counts = _counts(case, seed)
        offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        st["offsets"] = torch.from_numpy(offsets).cuda()
        if op == "product":
            st["x"], st["xs"] = _fp8((R, K), g), _scales((R, _up(K, BLOCK)), g, 117, 121)
            st["w"], st["ws"] = _fp8((E, N, K), g), _scales((E, _up(N, BLOCK), _up(K, BLOCK)), g, 112, 116)
            st["y"] = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
            live = np.nonzero(counts)[0]
            _, _, at, most = _padded(counts[live], 1)
            st["live"], st["at"] = torch.from_numpy(live).cuda(), torch.from_numpy(at).cuda()
            st["back"] = torch.from_numpy(np.nonzero(at.reshape(-1) < R)[0]).cuda()
        else:
            _, start, at, most = _padded(counts, BLOCK)
            B = int(start[-1])
            st["at"] = torch.from_numpy(at).cuda()
            valid = np.zeros(B * BLOCK, dtype=bool)
            for e in range(E):
                valid[start[e] * BLOCK:start[e] * BLOCK + counts[e]] = True
            valid = torch.from_numpy(valid).cuda()
            for n, rows in (("y", N), ("x", K)):
                q = _fp8((rows, B * BLOCK), g)
                q.view(torch.uint8)[:, ~valid] = 0
                st[n], st[n + "s"] = q, _scales((B, rows), g, 114, 118)
            st["dw"] = torch.empty(E, N, K, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _scale_of(amax):
    """The exponent e of the smallest 2^e with amax / 2^e <= 448 = 1.75 * 2^8."""
    m, ex = torch.frexp(amax)
    return torch.where(amax > 0, ex - 9 + (m > 0.875).int(), 0).clamp(-127, 127)


def _route_plain(st):
    c = st["case"]
    x = st["logits"].float()
    T, E, k = c["tokens"], c["experts"], c["k"]
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
        choice = s
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
        choice = x                                   # the same order
    if st["bias"] is not None:
        choice = choice + st["bias"]
    if c["groups"] > 1:
        by = choice.view(T, c["groups"], -1)
        best = torch.sort(by, dim=2, descending=True).values[..., :c["group_top"]].sum(2)
        stay = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        open_ = torch.zeros(T, c["groups"], dtype=torch.bool, device=x.device).scatter_(1, stay, True)
        choice = choice.masked_fill(~open_.repeat_interleave(E // c["groups"], 1), -torch.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    picked = torch.gather(s, 1, ids)
    w = picked / picked.sum(1, keepdim=True) if c["renorm"] else picked
    out = dict(ids=ids.int(), weights=w)
    if c["backward"]:
        gr = st["grad"]
        gs = (gr - (gr * w).sum(1, keepdim=True)) / picked.sum(1, keepdim=True) if c["renorm"] else gr
        full = torch.zeros_like(x).scatter_(1, ids, gs)
        gx = full * s * (1 - s) if c["score"] == "sigmoid" else s * (full - (full * s).sum(1, keepdim=True))
        out["grad_logits"] = gx.to(st["logits"].dtype)
    return out


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "route":
        return _route_plain(st)
    if op == "combine":
        offsets, slots, pos = _group(st["ids"], c["experts"])
        y = st["y"].float()
        rows = y[pos.long()]
        out = dict(offsets=offsets, slots=slots, pos=pos, out=(rows * st["weights"][..., None]).sum(1).bfloat16())
        if c["backward"]:
            gr = st["grad"].float()
            out["grad_weights"] = (rows * gr[:, None]).sum(2)
            gy = torch.empty_like(st["y"])
            gy[pos.reshape(-1).long()] = (gr[:, None] * st["weights"][..., None]).bfloat16().reshape(gy.shape)
            out["grad_y"] = gy
        return out
    if op in ("rows", "cols"):
        k, d = c["k"], c["hidden"]
        x = st["x"].float()[st["slots"].long() // k]
        if op == "rows":
            x = torch.nn.functional.pad(x, (0, -d % BLOCK)).view(x.shape[0], -1, BLOCK)
            e = _scale_of(x.abs().amax(2))
            q = torch.ldexp(x, -e[..., None]).view(x.shape[0], -1)[:, :d]
            return dict(q=q.to(F8), scales=(e + 127).to(torch.uint8))
        x = torch.cat([x, torch.zeros_like(x[:1])])[st["place"]].view(-1, BLOCK, d)
        e = _scale_of(x.abs().amax(1))
        q = torch.ldexp(x, -e[:, None]).view(-1, d).t().contiguous()
        return dict(q=q.to(F8), scales=((e + 127) * st["used"][:, None]).to(torch.uint8))
    if op == "blocks":
        w = st["w"].float()
        E, N, K = w.shape
        w = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK)).view(E, _up(N, BLOCK), BLOCK, _up(K, BLOCK), BLOCK)
        e = _scale_of(w.abs().amax((2, 4)))
        q = torch.ldexp(w, -e[:, :, None, :, None]).view(E, _up(N, BLOCK) * BLOCK, -1)[:, :N, :K].to(F8)
        s = (e + 127).to(torch.uint8)
        qt = q.view(torch.uint8).transpose(1, 2).contiguous().view(F8)
        return dict(q=q.contiguous(), scales=s, q_t=qt, scales_t=s.transpose(1, 2).contiguous())
    if op == "product":
        return _product(st, torch.float32).bfloat16()
    return _wgrad(st)


def _values(q, s, dt):
    """Rows of FP8 values with a scale for each 128 of a row."""
    return q.to(dt) * torch.exp2(s.to(dt) - 127).repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _product(st, dt):
    c = st["case"]
    x = _values(st["x"], st["xs"], dt)
    x = torch.cat([x, torch.zeros_like(x[:1])])[st["at"]]
    ws = st["ws"][st["live"]].repeat_interleave(BLOCK, 1)[:, :c["out"]]
    w = _values(st["w"].view(torch.uint8)[st["live"]].view(F8), ws, dt)
    return torch.bmm(x, w.transpose(1, 2)).view(-1, c["out"])[st["back"]]


def _wgrad(st):
    E, most = st["at"].shape

    def operand(q, s):
        v = q.float().view(q.shape[0], -1, BLOCK) * torch.exp2(s.t().float() - 127)[..., None]
        v = torch.cat([v, torch.zeros_like(v[:, :1])], 1)[:, st["at"].reshape(-1)]
        return v.view(q.shape[0], E, most * BLOCK).transpose(0, 1)

    return torch.bmm(operand(st["y"], st["ys"]), operand(st["x"], st["xs"]).transpose(1, 2))


# ------------------------------------------------------------------ the operators
def _own(st):
    ns, handle = _lib()
    h = handle.value
    c = st["case"]
    op = c["op"]
    if op == "route":
        score = ns.SCORE_SIGMOID if c["score"] == "sigmoid" else ns.SCORE_SOFTMAX
        ns.muon_moe_route(h, st["logits"], st["ids"], st["weights"], score=score, bias=st["bias"], groups=c["groups"],
                          top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"])
        out = dict(ids=st["ids"], weights=st["weights"])
        if c["backward"]:
            ns.muon_moe_route_backward(h, st["logits"], st["ids"], st["grad"], st["grad_logits"], score=score,
                                       renormalize=c["renorm"])
            out["grad_logits"] = st["grad_logits"]
        return out
    if op == "combine":
        offsets, slots, pos = st["plan"]
        ns.muon_moe_plan(h, st["ids"], offsets, slots, pos)
        ns.muon_moe_combine(h, st["y"], pos, st["weights"], st["out"])
        out = dict(offsets=offsets, slots=slots, pos=pos, out=st["out"])
        if c["backward"]:
            ns.muon_moe_combine_backward(h, st["grad"], st["y"], pos, st["weights"], st["grad_y"], st["grad_w"])
            out["grad_weights"], out["grad_y"] = st["grad_w"], st["grad_y"]
        return out
    if op == "rows":
        ns.muon_fp8_quantize_rows(h, st["x"], st["q"], st["s"], pos=st["pos"])
        return dict(q=st["q"], scales=st["s"])
    if op == "cols":
        ns.muon_fp8_quantize_cols(h, st["x"], st["offsets"], st["q"], st["s"], slots=st["slots"], top_k=c["k"])
        return dict(q=st["q"], scales=st["s"])
    if op == "blocks":
        ns.muon_fp8_quantize_blocks(h, st["w"], st["q"], st["s"], st["qt"], st["st"])
        return dict(q=st["q"], scales=st["s"], q_t=st["qt"], scales_t=st["st"])
    if op == "product":
        ns.muon_fp8_grouped_matmul(h, st["x"], st["xs"], st["w"], st["ws"], st["offsets"], st["y"])
        return st["y"]
    ns.muon_fp8_grouped_wgrad(h, st["y"], st["ys"], st["x"], st["xs"], st["offsets"], st["dw"])
    return st["dw"]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        el = 4 if case["dtype"] == "float32" else 2
        fwd, bwd = T * E * el + T * k * 8, 0
        if case["backward"]:
            bwd = T * E * el + T * k * 8 + (T * E * el if case["score"] == "softmax" and not case["renorm"] else T * k * el)
        return dict(bytes=fwd + bwd, flops=T * E * (8 if case["backward"] else 4))
    if op == "blocks":
        n = case["experts"] * case["rows"] * case["cols"]
        return dict(bytes=n * ((4 if case["dtype"] == "float32" else 2) + 2), flops=3 * n)
    if op == "combine":
        T, d, k = case["tokens"], case["hidden"], case["k"]
        n = T * k * d * 2 + T * d * 2 + T * k * 16
        if case["backward"]:
            n += 2 * T * k * d * 2 + T * d * 2 + T * k * 12
        return dict(bytes=n, flops=2 * T * k * d * (3 if case["backward"] else 1))
    if op in ("rows", "cols"):
        T, d, k = case["tokens"], case["hidden"], case["k"]
        return dict(bytes=T * d * 2 + T * k * (d + _up(d, BLOCK)) + T * k * 4, flops=3 * T * d)
    E, N, K, R = case["active"], case["out"], case["hidden"], case["rows"]
    live = min(E, R)
    if op == "product":
        return dict(bytes=R * K + live * N * K + 2 * R * N, flops=2 * R * N * K)
    return dict(bytes=R * (N + K) + 4 * case["experts"] * N * K, flops=2 * R * N * K)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x = st["logits"].double().cpu().numpy()
        T, E = x.shape
        k = case["k"]
        if case["score"] == "sigmoid":
            s = 1 / (1 + np.exp(-x))
        else:
            s = np.exp(x - x.max(1, keepdims=True))
            s /= s.sum(1, keepdims=True)
        c = (s if case["score"] == "sigmoid" else x) + (0.0 if st["bias"] is None else st["bias"].double().cpu().numpy())
        if case["groups"] > 1:
            v = c.reshape(T, case["groups"], -1)
            best = -np.sort(-v, axis=2)[..., :case["group_top"]].sum(2)
            order = np.argsort(-best, axis=1, kind="stable")[:, case["top_groups"]:]
            np.put_along_axis(v, order[..., None], -np.inf, 1)
            c = v.reshape(T, E)
        ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
        p = np.take_along_axis(s, ids, 1)
        total = p.sum(1, keepdims=True)
        w = p / total if case["renorm"] else p
        out = dict(ids=None, weights=w)
        if case["backward"]:
            gr = st["grad"].double().cpu().numpy()
            if case["renorm"]:
                gr = (gr - (gr * w).sum(1, keepdims=True)) / total
            gx = np.zeros_like(x)
            if case["score"] == "sigmoid":
                np.put_along_axis(gx, ids, gr * p * (1 - p), 1)
            else:
                gx -= s * (gr * p).sum(1, keepdims=True)
                np.put_along_axis(gx, ids, np.take_along_axis(gx, ids, 1) + gr * p, 1)
            out["grad_logits"] = gx
        return out
    if op == "combine":
        pos, w = st["pos"].long(), st["weights"].double()
        T, k = pos.shape
        out = torch.zeros(T, case["hidden"], dtype=torch.float64, device="cuda")
        gr = st["grad"].double()
        gw = torch.empty_like(w)
        gy = torch.empty(T * k, case["hidden"], dtype=torch.float64, device="cuda")
        for j in range(k):
            y = st["y"][pos[:, j]].double()
            out += y * w[:, j, None]
            gw[:, j] = (y * gr).sum(1)
            gy[pos[:, j]] = gr * w[:, j, None]
        res = dict(offsets=None, slots=None, pos=None, out=out)
        return dict(res, grad_weights=gw, grad_y=gy) if case["backward"] else res

    def power(amax):
        e = torch.ceil(torch.log2(amax / 448))
        return torch.where(amax > 0, e, torch.zeros_like(e))

    if op == "rows":
        x = st["x"].double()
        q = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for b in range(0, x.shape[1], BLOCK):
            v = x[:, b:b + BLOCK]
            q[:, b:b + BLOCK] = v / torch.exp2(power(v.abs().amax(1, keepdim=True)))
        out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            out[st["pos"][:, j].long()] = q
        return dict(q=out, scales=None)
    if op == "cols":
        slots, off = st["slots"].long().cpu().numpy(), st["offsets"].cpu().numpy()
        out, at = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"), 0
        for e in range(case["experts"]):
            for b in range(off[e], off[e + 1], BLOCK):
                rows = torch.from_numpy(slots[b:min(b + BLOCK, off[e + 1])] // case["k"]).cuda()
                v = st["x"][rows].double()
                out[:, at:at + len(rows)] = (v / torch.exp2(power(v.abs().amax(0, keepdim=True)))).t()
                at += BLOCK
        return dict(q=out, scales=None)
    if op == "blocks":
        E, N, K = st["w"].shape
        if E * N * K > 1 << 30:
            return None
        q = torch.empty(E, N, K, dtype=torch.float64, device="cuda")
        for n in range(0, N, BLOCK):
            for b in range(0, K, BLOCK):
                v = st["w"][:, n:n + BLOCK, b:b + BLOCK].double()
                q[:, n:n + BLOCK, b:b + BLOCK] = v / torch.exp2(power(v.abs().amax((1, 2), keepdim=True)))
        return dict(q=q, scales=None, q_t=q.transpose(1, 2), scales_t=None)
    off = st["offsets"].cpu().numpy()
    N, K = case["out"], case["hidden"]
    if 2.0 * case["rows"] * N * K > 4e12:
        return None
    if op == "product":
        y = torch.empty(case["rows"], N, dtype=torch.float64, device="cuda")
        for e in np.nonzero(np.diff(off))[0]:
            x = _values(st["x"][off[e]:off[e + 1]], st["xs"][off[e]:off[e + 1]], torch.float64)
            w = _values(st["w"][e], st["ws"][e].repeat_interleave(BLOCK, 0)[:N], torch.float64)
            y[off[e]:off[e + 1]] = x @ w.t()
        return y
    if case["experts"] * N * K > 1 << 31:
        return None
    dw, at = torch.zeros(case["experts"], N, K, dtype=torch.float64, device="cuda"), 0
    for e in range(case["experts"]):
        n = _up(int(off[e + 1] - off[e]), BLOCK)
        for b in range(at, at + n):
            cols = slice(b * BLOCK, (b + 1) * BLOCK)
            dy = st["y"][:, cols].double() * torch.exp2(st["ys"][b].double() - 127)[:, None]
            x = st["x"][:, cols].double() * torch.exp2(st["xs"][b].double() - 127)[:, None]
            dw[e] += dy @ x.t()
        at += n
    return dw
