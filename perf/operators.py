"""Measured cases of the operators that train a routed Mixture-of-Experts layer.

Five operators, each with its directions:

  dispatch    tokens laid out in expert order, from bf16/fp32 rows or from an
              e4m3 checkpoint of them; its gradient sums a token's rows and
              adds what the router's logits pass back
  combine     expert rows back to tokens with the routing weights applied, and
              its gradient (rows and weights)
  swiglu      h = silu(g) * u with g, u kept as e4m3 checkpoints (1 x 128
              blocks), and the gradient computed from the checkpoints
  route       the gradient of top-k routing: logits, router weight, bias
  product     one product per expert over its rows: forward, gradient of the
              rows, gradient of the weights

``own = False`` computes the plain forms with elementary torch operations in 32
bits; ``own = True`` calls the framework. Row i = (token t, slot k) with
i = t*K + k; ``inv[t, k]`` is its place in expert order, -1 for a dropped pair.
"""

import functools
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one decoded token of the full-size layer: launch latency
        _rows("dispatch_1tok", "dispatch", T=1, K=8, E=384, H=4096),
        # backward pass of a 4096-token step: x comes back from its 8-bit checkpoint in expert order; some
        # pairs are dropped
        _rows("dispatch_ckpt_4096", "dispatch", T=4096, K=8, E=384, H=4096, src="e4m3", drop=True),
        # the same step's gradient of x: eight rows per token and the router's share
        _rows("dispatch_bwd_4096", "dispatch_bwd", T=4096, K=8, E=384, H=4096, router=True),
        # a small layer with fp32 expert rows and an odd token count
        _rows("combine_1001", "combine", T=1001, K=4, E=48, H=512, src="fp32", drop=True),
        # gradient of the weighted combine of a 4096-token step
        _rows("combine_bwd_4096", "combine_bwd", T=4096, K=8, E=384, H=4096),
        # the activation of a 4095-token step, with its 8-bit checkpoint
        _swiglu("swiglu_4095", "swiglu", T=4095, K=8, E=384, I=2048),
        # its gradient, with the routing weights inside (nothing of the down product is kept)
        _swiglu("swiglu_bwd_4096", "swiglu_bwd", T=4096, K=8, E=384, I=2048, weighted=True),
        # router gradient of a few sequences' last tokens: latency
        _route("route_bwd_37", T=37, K=8, E=384, H=4096),
        # router gradient of a 4096-token step under the Zipf prior
        _route("route_bwd_4096", T=4096, K=8, E=384, H=4096),
        # gate/up of a short batch on one rank's 48 of 384 experts: reading the weights
        _product("product_333", "product", P=333, E=48, n_in=4096, n_out=4096, skew=1.1),
        # gradient of the rows through gate/up: one rank of eight, 4096 tokens each
        _product("product_dgrad_32768", "product_dgrad", P=32768, E=48, n_in=4096, n_out=4096, skew=0.0),
        # gradient of the gate/up weights of the same step, kept in fp32
        _product("wgrad_32768", "wgrad", P=32768, E=48, n_in=4096, n_out=4096, skew=0.0, src="fp32"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["dispatch", "dispatch_bwd", "combine", "combine_bwd", "swiglu", "swiglu_bwd", "route_bwd",
                     "product", "product_dgrad", "wgrad"])
    T, K = log_int(1, 4096), rng.randint(1, 8)
    E = max(K, log_int(4, 384))
    wide = 128 * log_int(2, 32)
    if op in ("dispatch", "dispatch_bwd", "combine", "combine_bwd"):
        src = rng.choice(["bf16", "bf16", "fp32"] + (["e4m3"] if op == "dispatch" else []))
        return _rows(None, op, T=T, K=K, E=E, H=wide, src=src, drop=T >= 8 and rng.random() < 0.3,
                     router=op == "dispatch_bwd" and rng.random() < 0.5)
    if op in ("swiglu", "swiglu_bwd"):
        return _swiglu(None, op, T=T, K=K, E=E, I=128 * log_int(1, 16), drop=T >= 8 and rng.random() < 0.3,
                       weighted=op == "swiglu_bwd" and rng.random() < 0.7)
    if op == "route_bwd":
        return _route(None, T=T, K=K, E=E, H=wide)
    P = log_int(1, 16384)
    return _product(None, op, P=P, E=log_int(1, 48), n_in=128 * log_int(1, 32), n_out=128 * log_int(1, 32),
                    skew=rng.choice([0.0, 1.1]) if P <= 4096 else 0.0,
                    src=rng.choice(["bf16", "fp32"]) if op == "wgrad" else "bf16")


def _case(name, **kw):
    return dict(kw) if name is None else dict(kw, name=name)


def _rows(name, op, T, K, E, H, src="bf16", drop=False, router=False):
    return _case(name, op=op, T=T, K=K, E=E, H=H, src=src, drop=drop, router=router)


def _swiglu(name, op, T, K, E, I, drop=False, weighted=False):
    return _case(name, op=op, T=T, K=K, E=E, I=I, drop=drop, weighted=weighted)


def _route(name, T, K, E, H):
    return _case(name, op="route_bwd", T=T, K=K, E=E, H=H)


def _product(name, op, P, E, n_in, n_out, skew, src="bf16"):
    """n_in, n_out: the forward product's; out [P, n_out] = a [P, n_in] W[e]^T, W [E, n_out, n_in]."""
    return _case(name, op=op, P=P, E=E, n_in=n_in, n_out=n_out, skew=skew, src=src)


# ------------------------------------------------------------------ inputs --

@functools.lru_cache(maxsize=None)
def _layer(H, E, K, I):
    """The layer a training program keeps (its context), one per configuration."""
    import mixture_experts_layer_24_b200 as M
    return M.MoeLayer(H, E, K, I)


def _randn(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def _routing(gen, T, K, E, drop):
    """Top-k of logits under a Zipf(1.1) prior and the permutation of the kept pairs."""
    prior = -1.1 * torch.log(1.0 + torch.randperm(E, generator=gen, device=DEV).float())
    logits = torch.randn(T, E, generator=gen, device=DEV) * 1.28 + prior
    top = torch.topk(logits, K, dim=1)
    w = torch.softmax(top.values, dim=1).contiguous()
    idx = top.indices
    key = idx.clone()
    if drop:  # one pair in sixteen names no expert, and so does every pair of one token
        key[torch.rand(T, K, generator=gen, device=DEV) < 1 / 16] = E
        key[T // 2] = E
    flat = key.reshape(-1)
    order = torch.argsort(flat, stable=True)
    n = int((flat < E).sum())
    inv = torch.empty(T * K, dtype=torch.int64, device=DEV)
    inv[order] = torch.arange(T * K, device=DEV)
    inv[flat >= E] = -1
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    return {"idx": idx.to(torch.int32).contiguous(), "w": w, "inv": inv.to(torch.int32).view(T, K), "n": n,
            "offsets": _offsets(counts), "perm_src": (order // K).to(torch.int32), "perm_k": (order % K).to(torch.int32)}


def _offsets(counts):
    return torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).to(torch.int32)


def _quant(v):
    """e4m3 codes and scales of 1 x 128 blocks, in 32 bits."""
    b = v.float().view(*v.shape[:-1], -1, 128)
    amax = b.abs().amax(-1)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    return (b / s[..., None]).view(v.shape).to(F8), s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, op = case, case["op"]
    st = {"op": op, "case": c}
    if op in ("product", "product_dgrad", "wgrad"):
        P, E, n_in, n_out = c["P"], c["E"], c["n_in"], c["n_out"]
        p = (1.0 + torch.randperm(E, generator=gen, device=DEV).double()) ** -c["skew"]
        pick = torch.multinomial(p, P, replacement=True, generator=gen)
        counts = torch.bincount(pick, minlength=E)
        st.update(offsets=_offsets(counts), most=int(counts.max()))
        if op == "wgrad":
            st.update(a=_randn(gen, P, n_in), dy=_randn(gen, P, n_out, std=0.01))
        else:
            st.update(a=_randn(gen, P, n_in if op == "product" else n_out),
                      w=_randn(gen, E * n_out, n_in, std=0.02).view(E, n_out, n_in))
        if own:
            wide = max(n_in, n_out)
            st["layer"] = _layer(min(8192, wide), E, 1, min(8192, wide))
        return st
    T, K, E = c["T"], c["K"], c["E"]
    st.update(_routing(gen, T, K, E, c.get("drop", False)))
    P = T * K
    if op == "route_bwd":
        st.update(x=_randn(gen, T, c["H"]), dw=_randn(gen, T, K, std=0.1, dtype=torch.float32))
    elif op in ("swiglu", "swiglu_bwd"):
        I = c["I"]
        gu = _randn(gen, P, 2 * I, std=1.3)
        bf = functools.partial(torch.zeros, dtype=torch.bfloat16, device=DEV)
        if op == "swiglu":
            st.update(gu=gu, out=(bf(P, I), torch.zeros(P, 2 * I, dtype=torch.uint8, device=DEV),
                                  torch.zeros(P, 2 * I // 128, device=DEV)))
        else:
            q, s = _quant(gu)
            st.update(q=q.view(torch.uint8), s=s, dh=_randn(gen, P, I, std=0.02),
                      out=(bf(P, 2 * I), bf(P, I) if c["weighted"] else None))
    else:
        H, dt = c["H"], TYPES.get(c["src"], torch.bfloat16)
        if op == "dispatch":
            x = _randn(gen, T, H, dtype=dt)
            if c["src"] == "e4m3":
                q, st["s"] = _quant(x)
                x = q.view(torch.uint8)
            st.update(x=x, out=torch.zeros(P, H, dtype=dt, device=DEV))
        elif op == "dispatch_bwd":
            st.update(rows=_randn(gen, P, H, std=0.02, dtype=dt))
            if c["router"]:
                st.update(dl=_randn(gen, T, K, std=0.01, dtype=torch.float32),
                          wr=_randn(gen, E, H, std=0.02, dtype=torch.float32))
        elif op == "combine":
            st.update(rows=_randn(gen, P, H, dtype=dt))
        else:
            st.update(rows=_randn(gen, P, H, dtype=dt), dout=_randn(gen, T, H, std=0.02, dtype=dt),
                      out=torch.zeros(P, H, dtype=dt, device=DEV))
    if own:
        st["layer"] = _layer(c.get("H", 256), E, K, c.get("I", 256))
    return st


# --------------------------------------------------------------------- run --

def run(st):
    return _framework(st) if own else _plain(st)


def _framework(st):
    op, c, L = st["op"], st["case"], st["layer"]
    if op == "dispatch":
        return L.dispatch(st["x"], st["inv"], x_scales=st.get("s"), out=st["out"])
    if op == "dispatch_bwd":
        if c["router"]:
            return L.dispatch_bwd(st["rows"], st["inv"], dlogit=st["dl"], topk_idx=st["idx"], w_router=st["wr"])
        return L.dispatch_bwd(st["rows"], st["inv"])
    if op == "combine":
        return L.combine_weighted(st["rows"], st["w"], st["inv"])
    if op == "combine_bwd":
        return L.combine_weighted_bwd(st["dout"], st["rows"], st["w"], st["inv"], out=st["out"])
    if op == "swiglu":
        h, q, s = L.swiglu_ckpt(st["gu"], st["inv"], out=st["out"])
        return h, q.view(F8), s
    if op == "swiglu_bwd":
        w = st["w"] if c["weighted"] else None
        return L.swiglu_ckpt_bwd(st["q"], st["s"], st["dh"], topk_w=w, inv=st["inv"], out=st["out"])
    if op == "route_bwd":
        return L.route_bwd(st["x"], st["w"], st["dw"], st["offsets"], st["perm_src"], st["perm_k"])
    if op == "wgrad":
        return L.expert_wgrad(st["dy"], st["a"], st["offsets"], dtype=TYPES[c["src"]])
    return L.expert_product(st["a"], st["w"], st["offsets"], transposed=op == "product_dgrad")


def _gathered(rows, inv):
    """rows[inv] in 32 bits, zeros for dropped pairs: [T, K, H]."""
    g = rows.float()[inv.clamp(min=0).long()]
    return g * (inv >= 0)[..., None]


def _weighted_places(st):
    """Token and place of each kept pair."""
    t, k = (st["inv"] >= 0).nonzero(as_tuple=True)
    return t, k, st["inv"][t, k].long()


def _padded(rows, st):
    """Each expert's rows in 32 bits, padded with zeros to the longest: [E, most, n]."""
    at = st["offsets"][:-1, None] + torch.arange(st["most"], device=DEV)
    kept = at < st["offsets"][1:, None]
    return rows.float()[at.clamp(max=rows.shape[0] - 1).long()] * kept[..., None], kept


def _plain(st):
    op, c, inv = st["op"], st["case"], st.get("inv")
    if op == "dispatch":
        x = st["x"]
        if c["src"] == "e4m3":
            b = x.view(F8).float().view(x.shape[0], -1, 128) * st["s"][..., None]
            x = b.view(x.shape).to(torch.bfloat16)
        st["out"][:st["n"]] = x[st["perm_src"][:st["n"]].long()]
        return st["out"]
    if op == "dispatch_bwd":
        dx = _gathered(st["rows"], inv).sum(1)
        if c["router"]:
            dx += (st["dl"][..., None] * st["wr"][st["idx"].long()]).sum(1)
        return dx.to(st["rows"].dtype)
    if op == "combine":
        return (_gathered(st["rows"], inv) * st["w"][..., None]).sum(1).to(st["rows"].dtype)
    if op == "combine_bwd":
        dw = (_gathered(st["rows"], inv) * st["dout"].float()[:, None]).sum(-1)
        t, k, p = _weighted_places(st)
        st["out"][p] = (st["w"][t, k, None] * st["dout"].float()[t]).to(st["out"].dtype)
        return st["out"], dw
    if op == "swiglu":
        n, (h, q, s) = st["n"], st["out"]
        gu = st["gu"][:n].float()
        g, u = gu.chunk(2, dim=1)
        h[:n] = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
        code, s[:n] = _quant(gu)
        q[:n] = code.view(torch.uint8)
        return h, q.view(F8), s
    if op == "swiglu_bwd":
        n, (dgu, hw) = st["n"], st["out"]
        q = st["q"][:n].view(F8).float()
        g, u = (q.view(n, -1, 128) * st["s"][:n, :, None]).view(n, -1).chunk(2, dim=1)
        dh, sig, dw = st["dh"][:n].float(), torch.sigmoid(g), None
        h = g * sig * u
        if c["weighted"]:
            t, k, p = _weighted_places(st)
            dw = torch.zeros_like(st["w"])
            dw[t, k] = (dh * h).sum(1)[p]
            w = torch.zeros(n, 1, device=DEV)
            w[p, 0] = st["w"][t, k]
            hw[:n] = (w * h).to(torch.bfloat16)
            dh = w * dh
        dgu[:n] = torch.cat((dh * u * sig * (1 + g * (1 - sig)), dh * g * sig), 1).to(torch.bfloat16)
        return dgu, hw, dw
    if op == "route_bwd":
        w, dw = st["w"], st["dw"]
        dl = w * (dw - (w * dw).sum(1, keepdim=True))
        full = torch.zeros(c["T"], c["E"], device=DEV).scatter_(1, st["idx"].long(), dl)
        return dl, full.t() @ st["x"].float(), full.sum(0)
    a, kept = _padded(st["a"], st)
    if op == "wgrad":
        dy, _ = _padded(st["dy"], st)
        return torch.bmm(dy.transpose(1, 2), a).to(TYPES[c["src"]])
    w = st["w"].float()
    return torch.bmm(a, w if op == "product_dgrad" else w.transpose(1, 2))[kept].to(torch.bfloat16)


# -------------------------------------------------------------------- work --

def work(case):
    c, op = case, case["op"]
    if op in ("product", "product_dgrad", "wgrad"):
        P, E, n_in, n_out = c["P"], c["E"], c["n_in"], c["n_out"]
        weights = E * n_in * n_out
        if op == "wgrad":
            weights *= 4 if c["src"] == "fp32" else 2
        else:
            weights = min(E, P) * n_in * n_out * 2  # at most the experts that have rows
        return {"bytes": weights + 2 * P * (n_in + n_out), "flops": 2 * P * n_in * n_out}
    T, K, E = c["T"], c["K"], c["E"]
    P = T * K
    if op in ("swiglu", "swiglu_bwd"):
        I = c["I"]
        ckpt = 2 * I + 4 * (2 * I // 128)
        if op == "swiglu":
            return {"bytes": P * (4 * I + 2 * I + ckpt), "flops": 8 * P * I}
        return {"bytes": P * (ckpt + 2 * I + 4 * I + (2 * I + 8 if c["weighted"] else 0)), "flops": 16 * P * I}
    H = c["H"]
    if op == "route_bwd":
        return {"bytes": 2 * T * H + 4 * E * H + 24 * P, "flops": 2 * P * H}
    size = 4 if c["src"] == "fp32" else 2
    if op == "dispatch":
        src = H + 4 * (H // 128) if c["src"] == "e4m3" else size * H
        return {"bytes": T * src + P * size * H + 4 * P, "flops": 0}
    if op == "dispatch_bwd":
        return {"bytes": (P + T) * size * H + 4 * P + (4 * min(E, P) * H + 8 * P if c["router"] else 0), "flops": P * H}
    if op == "combine":
        return {"bytes": (P + T) * size * H + 8 * P, "flops": 2 * P * H}
    return {"bytes": (2 * P + T) * size * H + 12 * P, "flops": 3 * P * H}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits. Loops over slots or experts keep the memory small."""
    st = prepare(case, seed)
    c, op = case, case["op"]
    f64 = torch.float64
    if op in ("product", "product_dgrad", "wgrad"):
        cut = st["offsets"].tolist()
        a = st["a"].to(f64)
        if op == "wgrad":
            dy = st["dy"].to(f64)
            return torch.stack([dy[i:j].t() @ a[i:j] for i, j in zip(cut, cut[1:])])
        return torch.cat([a[i:j] @ (m.to(f64) if op == "product_dgrad" else m.to(f64).t())
                          for i, j, m in zip(cut, cut[1:], st["w"])])
    T, K = c["T"], c["K"]
    inv, w = st["inv"].long(), st["w"].to(f64)
    if op == "route_bwd":
        dw = st["dw"].to(f64)
        dl = w * dw - w * (w * dw).sum(1, keepdim=True)
        x, full = st["x"].to(f64), torch.zeros(T, c["E"], dtype=f64, device=DEV)
        for k in range(K):
            full[torch.arange(T, device=DEV), st["idx"][:, k].long()] = dl[:, k]
        return dl, torch.einsum("te,th->eh", full, x), full.sum(0)
    P = T * K
    if op in ("swiglu", "swiglu_bwd"):
        I, live = c["I"], torch.zeros(P, dtype=torch.bool, device=DEV)
        live[inv[inv >= 0]] = True
        live = live[:, None]
        if op == "swiglu":
            gu = st["gu"].to(f64)
            g, u = gu[:, :I], gu[:, I:]
            h = torch.where(live, g / (1 + torch.exp(-g)) * u, 0.0)
            amax = gu.view(P, -1, 128).abs().amax(-1)
            s = torch.where(amax > 0, amax / 448, 1.0)
            q = (gu.view(P, -1, 128) / s[..., None]).view(P, 2 * I)
            return h, torch.where(live, q, 0.0), torch.where(live, s, 0.0)
        v = (st["q"].view(F8).to(f64).view(P, -1, 128) * st["s"].to(f64)[..., None]).view(P, 2 * I)
        g, u, dh = v[:, :I], v[:, I:], st["dh"].to(f64)
        e = 1 / (1 + torch.exp(-g))
        scale, dw, hw = torch.ones(P, 1, dtype=f64, device=DEV), None, None
        if c["weighted"]:
            scale = torch.zeros(P + 1, dtype=f64, device=DEV)
            scale[inv.reshape(-1)] = w.reshape(-1)  # dropped pairs land in the last place
            scale = scale[:P, None]
            dot = torch.nn.functional.pad((dh * g * e * u).sum(1), (0, 1))
            dot[P] = 0.0
            dw = dot[inv]
            hw = torch.where(live, scale * g * e * u, 0.0)
        dgu = torch.cat((scale * dh * u * (e + g * e * (1 - e)), scale * dh * g * e), 1)
        return torch.where(live, dgu, 0.0), hw, dw
    H = c["H"]
    if op == "dispatch":
        x = st["x"]
        if c["src"] == "e4m3":
            x = (x.view(F8).to(f64).view(T, -1, 128) * st["s"].to(f64)[..., None]).view(T, H)
        out = torch.zeros(P, H, dtype=f64, device=DEV)
        for k in range(K):
            out[inv[inv[:, k] >= 0, k]] = x[inv[:, k] >= 0].to(f64)
        return out
    acc, dy, dots = torch.zeros(T, H, dtype=f64, device=DEV), None, []
    if op == "combine_bwd":
        dy, dout = torch.zeros(P, H, dtype=f64, device=DEV), st["dout"].to(f64)
    for k in range(K):
        kept = (inv[:, k] >= 0)[:, None]
        y = torch.where(kept, st["rows"][inv[:, k].clamp(min=0)].to(f64), 0.0)
        if op == "dispatch_bwd":
            acc += y
            if c["router"]:
                acc += st["dl"][:, k, None].to(f64) * st["wr"][st["idx"][:, k].long()].to(f64)
        elif op == "combine":
            acc += w[:, k, None] * y
        else:
            dots.append((dout * y).sum(1))
            dy[inv[kept[:, 0], k]] = (w[:, k, None] * dout)[kept[:, 0]]
    return acc if op != "combine_bwd" else (dy, torch.stack(dots, 1))
