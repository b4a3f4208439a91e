"""The layer's operators around quantised experts, as cases that can be timed and checked.

Four operators, each in its plain form (elementary torch operations) and through
the package's entry points:

  route   scored routing: softmax or sigmoid scores, a balance bias, expert groups,
          top-k and renormalised weights (moe_route_scored)
  linear  int8 x int8 matrix product with a scale per token and per output
          channel (moe_linear_int8)
  ffn     the grouped gated FFN over int8 experts with int8 activations, and the
          combine that follows it (moe_grouped_ffn_w8a8, moe_combine)
  norm    the norms around a block: combine (or a dense block's output), norm after
          the block, gates, residual, norm before the next block, int8 codes for
          its products (moe_combine_norm, moe_residual_norm, moe_norm)

``own`` selects the form ``run`` takes.  Sizes are the repository's own (128
experts, hidden 2816, expert intermediate 704, top-8) or generic.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DEV = "cuda"
_LOWEST = torch.finfo(torch.float32).min


def _pkg():
    import moe_router_softmax_b200 as moe

    return moe


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step: 128 experts, softmax scores, balance bias
        {"name": "route_one_token", "op": "route", "T": 1, "E": 128, "k": 8, "score": "softmax", "bias": True,
         "n_group": 1, "topk_group": 1, "group_top": 1, "renorm": True, "scale": 1.0, "masked": 0},
        # a decode batch over an odd number of experts, three of them out of service
        {"name": "route_batch_odd", "op": "route", "T": 61, "E": 165, "k": 6, "score": "softmax", "bias": False,
         "n_group": 5, "topk_group": 3, "group_top": 1, "renorm": False, "scale": 1.5, "masked": 3},
        # a prefill chunk over 256 experts in 8 groups, sigmoid scores, balance bias
        {"name": "route_prefill_groups", "op": "route", "T": 8192, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "n_group": 8, "topk_group": 4, "group_top": 2, "renorm": True, "scale": 2.5, "masked": 0},
        # one token through a square projection
        {"name": "linear_one_token", "op": "linear", "T": 1, "N": 2816, "K": 2816, "out": "bf16"},
        # a ragged decode batch through an expert-sized gate and up projection
        {"name": "linear_batch_odd", "op": "linear", "T": 77, "N": 1409, "K": 2816, "out": "fp32"},
        # a prefill chunk through a wide projection
        {"name": "linear_prefill", "op": "linear", "T": 4096, "N": 8192, "K": 2816, "out": "bf16"},
        # one decode step of one sequence
        {"name": "ffn_one_token", "op": "ffn", "T": 1, "E": 128, "H": 2816, "I": 704, "k": 8},
        # a decode batch
        {"name": "ffn_batch", "op": "ffn", "T": 64, "E": 128, "H": 2816, "I": 704, "k": 8},
        # a prefill chunk of odd length
        {"name": "ffn_prefill_odd", "op": "ffn", "T": 2047, "E": 128, "H": 2816, "I": 704, "k": 8},
        # the end of one layer and the start of the next for one token
        {"name": "norm_one_token", "op": "norm", "kind": "combine", "T": 1, "H": 2816, "k": 8, "codes": False},
        # the norm before a block for a ragged batch, with the codes of the block's int8 products
        {"name": "norm_before_odd", "op": "norm", "kind": "before", "T": 1023, "H": 2816, "k": 0, "codes": True},
        # a prefill chunk: combine, norms, gates and residual
        {"name": "norm_prefill", "op": "norm", "kind": "combine", "T": 8192, "H": 2816, "k": 8, "codes": False},
        ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "linear", "ffn", "norm"])
    if op == "route":
        while True:
            n_group = rng.choice([1, 1, 2, 3, 4, 6, 8, 16])
            size = _log(rng, 2, 1024)
            if 8 <= n_group * size <= 1024:
                break
        E = n_group * size
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(32, topk_group * size, 1 + E // 4))
        T = min(_log(rng, 1, 8192), 8192 * 256 // E + 1)
        return {"op": op, "T": T, "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.6, "n_group": n_group, "topk_group": topk_group,
                "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 0.5, 2.5]),
                "masked": rng.choice([0, 0, 1, E // 8])}
    if op == "linear":
        while True:
            T, N, K = _log(rng, 1, 4096), _log(rng, 33, 8192), 16 * _log(rng, 4, 512)
            if T * N * K <= 4096 * 8192 * 2816:
                break
        return {"op": op, "T": T, "N": N, "K": K, "out": rng.choice(["bf16", "fp32"])}
    if op == "ffn":
        while True:
            T, E = _log(rng, 1, 2047), _log(rng, 4, 160)
            H, I, k = 64 * _log(rng, 2, 64), 64 * _log(rng, 1, 32), rng.randint(1, min(E, 12))
            if T * k * H * I <= 2047 * 8 * 2816 * 704 and E * H * I <= 128 * 2816 * 704:
                break
        return {"op": op, "T": T, "E": E, "H": H, "I": I, "k": k}
    kind = rng.choice(["combine", "dense", "before"])
    while True:
        T, H = _log(rng, 1, 8192), 64 * _log(rng, 1, 128)
        k = rng.randint(1, 12) if kind == "combine" else 0
        if T * H * (k + 1) <= 8192 * 2816 * 9:
            break
    return {"op": op, "kind": kind, "T": T, "H": H, "k": k, "codes": rng.random() < 0.6}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=_DEV)


def _activations(g, T, H):
    """Hidden states: unit variance with a few strong channels, tokens of unlike norms."""
    x = _randn(g, T, H) * torch.exp(0.3 * _randn(g, T, 1))
    strong = torch.rand(H, generator=g, device=_DEV) < 0.004
    return torch.where(strong, 8.0 * x, x).bfloat16()


def _codes(v):
    """int8 codes and the fp32 scale of each row."""
    s = v.abs().amax(-1) / 127.0
    return torch.clamp(torch.round(v / s[..., None]), -127, 127).to(torch.int8), s


def _weights(g, *shape):
    q = torch.randint(-127, 128, shape, generator=g, device=_DEV, dtype=torch.int8)
    s = 0.0004 * (0.5 + torch.rand(shape[:-1], generator=g, device=_DEV))
    return q, s


def _routes(g, T, E, k):
    """A token's k experts, and the routes grouped by expert."""
    lg = _randn(g, T, E) + 0.5 * _randn(g, 1, E)
    top = torch.topk(lg, k, dim=1)
    ids = top.indices.to(torch.int32).contiguous()
    w = torch.softmax(top.values, dim=1).contiguous()
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device=_DEV)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=_DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    i32 = torch.int32
    return {"w": w, "counts": counts.to(i32), "offsets": offsets.to(i32), "sorted": order.to(i32),
            "pos": pos.to(i32)}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": dict(case)}
    T = case["T"]
    if op == "route":
        E = case["E"]
        lg = 1.5 * _randn(g, T, E) + 0.4 * _randn(g, 1, E)
        bias = 0.05 * _randn(g, E) if case["bias"] or case["masked"] else None
        if bias is not None and not case["bias"]:
            bias.zero_()
        if case["masked"]:
            # experts out of service: some by their bias, some by every logit
            off = torch.randperm(E, generator=g, device=_DEV)[:case["masked"]]
            bias[off[::2]] = float("-inf")
            lg[:, off[1::2]] = float("-inf")
        st.update(logits=lg.contiguous(), bias=bias)
    elif op == "linear":
        xq, sx = _codes(_activations(g, T, case["K"]).float())
        wq, sw = _weights(g, case["N"], case["K"])
        st.update(xq=xq, sx=sx, wq=wq, sw=sw)
    elif op == "ffn":
        E, H, I = case["E"], case["H"], case["I"]
        xq, sx = _codes(_activations(g, T, H).float())
        # the layer's blobs, expert after expert: codes and scales of w13, then of w2
        parts = [(2 * I * H, torch.int8), (8 * I, torch.float32), (H * I, torch.int8), (4 * H, torch.float32)]
        stride = (sum(n for n, _ in parts) + 255) // 256 * 256
        home = torch.zeros((E, stride), dtype=torch.uint8, device=_DEV)
        views, at = [], 0
        for (n, dt), t in zip(parts, (*_weights(g, E, 2 * I, H), *_weights(g, E, H, I))):
            home[:, at:at + n] = t.reshape(E, -1).view(torch.uint8)
            views.append(home[:, at:at + n].view(dt))
            at += n
        st.update(xq=xq, sx=sx, home=home, q13=views[0].unflatten(1, (2 * I, H)), s13=views[1],
                  q2=views[2].unflatten(1, (H, I)), s2=views[3], **_routes(g, T, E, case["k"]))
        if own:
            moe = _pkg()
            st["layer"] = moe.MoeLayer(moe.MOE_W_INT8, E, H, I, home.view(-1), expert_bytes=stride)
            st["ws"] = torch.empty(moe.moe_grouped_ffn_w8a8_workspace(st["layer"], T, case["k"]), dtype=torch.uint8,
                                   device=_DEV)
            st["rows"] = torch.empty((T * case["k"], H), device=_DEV)
    else:
        H, k = case["H"], case["k"]
        st["next_w"] = (1.0 + 0.2 * _randn(g, H)).bfloat16()
        st["x"] = _activations(g, T, H)  # the block's input, carried past it
        if case["kind"] != "before":
            st["post_w"] = (0.5 + 0.1 * _randn(g, H)).bfloat16()
            st["gate_h"] = 1.0 + 0.1 * _randn(g, H)
            st["gate_t"] = torch.sigmoid(_randn(g, T))
        if case["kind"] == "dense":
            st["z"] = (0.1 * _randn(g, T, H)).bfloat16()
        if case["kind"] == "combine":
            st["rows"] = 0.1 * _randn(g, T * k, H)
            st["pos"] = torch.randperm(T * k, generator=g, device=_DEV).to(torch.int32)
            w = torch.rand((T, k), generator=g, device=_DEV) + 0.05
            st["w"] = (w / w.sum(1, keepdim=True)).contiguous()
            # a few routes were dropped by the router
            st["pos"][torch.rand(T * k, generator=g, device=_DEV) < 0.01] = -1
    return st


_EPS = 1e-6
_RES, _BLOCK = 0.75, 1.25  # residual and block scales of the norm cases


# ------------------------------------------------------------------ plain forms

def _plain_route(st):
    # in 64 bits: a choice next to a border decides an id
    c, logits = st["case"], st["logits"]
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    live = logits > _LOWEST
    l = torch.where(live, logits, torch.full_like(logits, float("-inf"))).double()
    if c["score"] == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.where(live, torch.exp(torch.where(l == m, torch.zeros_like(l), l - m)), torch.zeros_like(l))
        z = e.sum(1, keepdim=True)
        s = torch.where(z > 0, e / z, torch.zeros_like(e))
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    ch = s
    if st["bias"] is not None:
        live = live & (st["bias"] > _LOWEST)
        ch = s + st["bias"].double()
    none = torch.full_like(ch, float("-inf"))
    ch = torch.where(live, ch, none)
    if G > 1:
        best = torch.sort(ch.view(T, G, E // G), dim=2, descending=True, stable=True).values[:, :, :c["group_top"]]
        has = best[:, :, :1] > float("-inf")
        gs = torch.where(best > float("-inf"), best, torch.zeros_like(best)).sum(2)
        gs = torch.where(has[:, :, 0], gs, torch.full_like(gs, float("-inf")))
        keep = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        on = torch.zeros((T, G), dtype=torch.bool, device=logits.device).scatter_(1, keep, True)
        ch = torch.where(on.repeat_interleave(E // G, 1), ch, none)
    top = torch.sort(ch, dim=1, descending=True, stable=True)
    ids, taken = top.indices[:, :k], top.values[:, :k] > float("-inf")
    w = torch.where(taken, torch.gather(s, 1, ids), torch.zeros_like(s[:, :k]))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    ids = torch.where(taken, ids, torch.full_like(ids, -1))
    return {"ids": ids.to(torch.int32), "w": (w * c["scale"]).float()}


def _plain_linear(st):
    y = (st["xq"].float() @ st["wq"].float().t()) * st["sx"][:, None] * st["sw"]
    return {"y": y.bfloat16() if st["case"]["out"] == "bf16" else y}


def _plain_ffn(st):
    c = st["case"]
    T, H, I, k = c["T"], c["H"], c["I"], c["k"]
    # the experts that hold routes, each with its routes padded to the busiest one's
    act = torch.nonzero(st["counts"])[:, 0]
    n = st["counts"][act].long()
    j = torch.arange(int(n.max()), device=n.device)
    held = j < n[:, None]
    row = torch.where(held, st["offsets"][act].long()[:, None] + j, 0)
    token = st["sorted"][row].long() // k
    g = torch.bmm(st["xq"][token].float(), st["q13"][act].float().transpose(1, 2))
    g = g * st["sx"][token][:, :, None] * st["s13"][act][:, None, :]
    a, u = g[:, :, :I], g[:, :, I:]
    h = 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a))) * u
    s = h.abs().amax(2, keepdim=True) / 127.0
    q = torch.clamp(torch.round(h / torch.where(s > 0, s, 1.0)), -127, 127)
    o = torch.bmm(q, st["q2"][act].float().transpose(1, 2)) * s * st["s2"][act][:, None, :]
    rows = torch.empty((T * k, H), device=o.device)
    rows[row[held]] = o[held]
    y = (rows[st["pos"].long()].view(T, k, H) * st["w"][:, :, None]).sum(1)
    return {"y": y.bfloat16()}


def _plain_norm(st):
    c = st["case"]
    T, H, k = c["T"], c["H"], c["k"]
    out = {}
    x = st["x"].float()
    if c["kind"] != "before":
        if c["kind"] == "combine":
            pos = st["pos"].long()
            r = torch.where(pos[:, None] >= 0, st["rows"][pos.clamp(min=0)], torch.zeros_like(st["rows"]))
            z = (r.view(T, k, H) * st["w"][:, :, None]).sum(1)
        else:
            z = st["z"].float()
        z = z * torch.rsqrt((z * z).mean(1, keepdim=True) + _EPS) * st["post_w"].float()
        y = (_RES * x + _BLOCK * st["gate_t"][:, None] * st["gate_h"] * z).bfloat16()
        out["y"] = y
        x = y.float()
    # in 64 bits: a value next to a border decides a code
    x = x.double()
    n = x * torch.rsqrt((x * x).mean(1, keepdim=True) + _EPS) * st["next_w"].double()
    out["xn"] = n.bfloat16()
    if c["codes"]:
        s = n.abs().amax(1, keepdim=True) / 127.0
        q = torch.clamp(torch.round(n / torch.where(s > 0, s, 1.0)), -127, 127)
        out["values"] = (q * s).bfloat16()
    return out


# ------------------------------------------------------------------ the package's calls

def _own_route(st):
    moe, c = _pkg(), st["case"]
    score = moe.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else moe.MOE_SCORE_SIGMOID
    ids, w = moe.moe_route_scored(st["logits"], c["k"], bias=st["bias"], score=score, n_group=c["n_group"],
                                  topk_group=c["topk_group"], group_top=c["group_top"], renorm=c["renorm"],
                                  scale=c["scale"])
    return {"ids": ids, "w": w}


def _own_linear(st):
    dt = torch.bfloat16 if st["case"]["out"] == "bf16" else torch.float32
    return {"y": _pkg().moe_linear_int8(st["xq"], st["sx"], st["wq"], st["sw"], dtype=dt)}


def _own_ffn(st):
    moe = _pkg()
    rows = moe.moe_grouped_ffn_w8a8(st["layer"], st["xq"], st["sx"], st["case"]["k"], st["counts"], st["offsets"],
                                    st["sorted"], rows=st["rows"], ws=st["ws"])
    return {"y": moe.moe_combine(rows, st["pos"], st["w"])}


def _own_norm(st):
    moe, c = _pkg(), st["case"]
    if c["kind"] == "before":
        out = moe.moe_norm(st["x"], st["next_w"], eps=_EPS, codes=c["codes"])
    else:
        kw = dict(eps=_EPS, residual_scale=_RES, block_scale=_BLOCK, gate_h=st["gate_h"], gate_t=st["gate_t"],
                  next_weight=st["next_w"], codes=c["codes"])
        if c["kind"] == "combine":
            out = moe.moe_combine_norm(st["rows"], st["pos"], st["w"], st["x"], st["post_w"], **kw)
        else:
            out = moe.moe_residual_norm(st["z"], st["x"], st["post_w"], **kw)
    res = {}
    if out.y is not None:
        res["y"] = out.y
    res["xn"] = out.xn
    if c["codes"]:
        # codes and scales as the values they stand for (8 bits: bf16 holds what matters of them)
        res["values"] = torch.mul(out.xq, out.sx[:, None], out=torch.empty_like(out.xn))
    return res


_PLAIN = {"route": _plain_route, "linear": _plain_linear, "ffn": _plain_ffn, "norm": _plain_norm}
_OWN = {"route": _own_route, "linear": _own_linear, "ffn": _own_ffn, "norm": _own_norm}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        E, k = case["E"], case["k"]
        return {"bytes": 4 * T * E + (4 * E if case["bias"] or case["masked"] else 0) + 8 * T * k, "flops": 4 * T * E}
    if op == "linear":
        N, K = case["N"], case["K"]
        ob = 2 if case["out"] == "bf16" else 4
        return {"bytes": T * K + N * K + 4 * (T + N) + ob * T * N, "flops": 2 * T * N * K}
    if op == "ffn":
        E, H, I, k = case["E"], case["H"], case["I"], case["k"]
        # experts that T tokens of k experts each reach, at uniform popularity
        active = E * (1.0 - (1.0 - k / E) ** T)
        return {"bytes": int(active * (3 * H * I + 4 * (2 * I + H))) + T * H + 4 * T + 16 * T * k + 8 * E + 2 * T * H,
                "flops": 6 * T * k * H * I}
    H, k = case["H"], case["k"]
    b = 2 * T * H + 2 * H + 2 * T * H + (T * H + 4 * T if case["codes"] else 0)
    f = 5 * T * H
    if case["kind"] != "before":
        b += 2 * T * H + 6 * H + 4 * T + (4 * T * k * H + 8 * T * k if case["kind"] == "combine" else 2 * T * H)
        f += (8 + 2 * k) * T * H
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_route(case, st):
    T, E, k, G = case["T"], case["E"], case["k"], case["n_group"]
    l32 = st["logits"].cpu().numpy()
    ok = l32 > np.float32(_LOWEST)
    l = np.where(ok, l32, -np.inf).astype(np.float64)
    if case["score"] == "softmax":
        m = l.max(1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        s = np.exp(l - m)
        z = s.sum(1, keepdims=True)
        s = np.divide(s, z, out=np.zeros_like(s), where=z > 0)
    else:
        s = np.where(ok, 1.0 / (1.0 + np.exp(-np.where(ok, l, 0.0))), 0.0)
    c = s.copy()
    if st["bias"] is not None:
        b = st["bias"].cpu().numpy()
        ok = ok & (b > np.float32(_LOWEST))[None, :]
        c = c + np.where(np.isfinite(b), b, 0.0).astype(np.float64)
    c[~ok] = -np.inf
    t_all = np.arange(T)
    if G > 1:
        cg = c.reshape(T, G, E // G).copy()
        gs = np.zeros((T, G))
        dead = ~np.isfinite(cg).any(2)
        for _ in range(min(case["group_top"], E // G)):
            j = cg.argmax(2)
            v = np.take_along_axis(cg, j[:, :, None], 2)[:, :, 0]
            gs += np.where(np.isfinite(v), v, 0.0)
            np.put_along_axis(cg, j[:, :, None], -np.inf, 2)
        gs[dead] = -np.inf
        on = np.zeros((T, G), bool)
        for _ in range(case["topk_group"]):
            # dead groups may be kept: nothing is taken from them
            j = np.where(on, -np.inf, gs).argmax(1)
            on[t_all, j] = True
        c = np.where(np.repeat(on, E // G, 1), c, -np.inf)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for j in range(k):
        e = c.argmax(1)
        got = c[t_all, e] > -np.inf
        ids[got, j] = e[got]
        w[got, j] = s[t_all, e][got]
        c[t_all, e] = -np.inf
    if case["renorm"]:
        z = w.sum(1, keepdims=True)
        w = np.divide(w, z, out=np.zeros_like(w), where=z > 0)
    return {"ids": ids, "w": w * case["scale"]}


def _exact_ffn(case, st):
    q13, s13, q2, s2 = st["q13"], st["s13"], st["q2"], st["s2"]
    T, H, I, k = case["T"], case["H"], case["I"], case["k"]
    counts = st["counts"].tolist()
    y = torch.zeros((T, H), dtype=torch.float64, device=_DEV)
    wf = st["w"].double().flatten()
    lo = 0
    for e, n in enumerate(counts):
        routes = st["sorted"][lo:lo + n].long()
        lo += n
        if n == 0:
            continue
        t = torch.div(routes, k, rounding_mode="floor")
        x = st["xq"][t].double() * st["sx"][t].double()[:, None]
        w13 = q13[e].double() * s13[e].double()[:, None]
        gate, up = x @ w13[:I].t(), x @ w13[I:].t()
        h = gate * up * (1.0 - 1.0 / (1.0 + torch.exp(2.0 * (2.0 / math.pi) ** 0.5 * (gate + 0.044715 * gate ** 3))))
        s = h.abs().amax(1, keepdim=True) / 127.0
        code = torch.where(s > 0, torch.round(h / torch.where(s > 0, s, 1.0)), 0.0).clamp(-127, 127)
        row = (code * s) @ (q2[e].double() * s2[e].double()[:, None]).t()
        y.index_add_(0, t, row * wf[routes][:, None])
    return {"y": y}


def _exact_norm(case, st):
    T, H, k = case["T"], case["H"], case["k"]
    res = {}
    x = st["x"].double()
    if case["kind"] != "before":
        if case["kind"] == "dense":
            z = st["z"].double()
        else:
            z = torch.zeros((T, H), dtype=torch.float64, device=_DEV)
            pos = st["pos"].view(T, k).long()
            for j in range(k):
                ok = pos[:, j] >= 0
                z[ok] += st["w"][ok, j].double()[:, None] * st["rows"][pos[ok, j]].double()
        z = z / torch.sqrt(z.square().sum(1, keepdim=True) / H + _EPS)
        y = st["gate_h"].double() * st["gate_t"].double()[:, None] * (_BLOCK * z * st["post_w"].double()) + _RES * x
        res["y"] = y
        x = y.bfloat16().double()  # the next block reads what is stored
    n = x / torch.sqrt(x.square().sum(1, keepdim=True) / H + _EPS) * st["next_w"].double()
    res["xn"] = n
    if case["codes"]:
        s = n.abs().amax(1, keepdim=True) / 127.0
        res["values"] = torch.where(s > 0, torch.round(n / torch.where(s > 0, s, 1.0)), 0.0).clamp(-127, 127) * s
    return res


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "linear":
        x = st["xq"].double() * st["sx"].double()[:, None]
        return {"y": x @ (st["wq"].double() * st["sw"].double()[:, None]).t()}
    if op == "ffn":
        return _exact_ffn(case, st)
    return _exact_norm(case, st)
