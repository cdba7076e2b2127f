"""The operators around the optimizer step, measured: the embedding, the
language-model head's loss and the experts' products, forward and backward.

The optimizer updates an embedding and a head (AdamW) and experts' matrices
(Muon); these are the calls that read those weights and make their gradients.
``own`` chooses between the plain torch form and the library's kernels; both
take the same inputs and return the same outputs.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
IGNORE = -100


# --------------------------------------------------------------------------
# The cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token's row at the start of a decoding step: latency alone
        dict(name="lookup_one_token", op="lookup", vocab=163840, dim=7168, tokens=1, table="bf16", out="bf16", pads=0.0),
        # a training batch read from the fp32 master table, rounded to the compute type
        dict(name="lookup_master_batch", op="lookup", vocab=163840, dim=7168, tokens=32768, table="fp32", out="bf16",
             pads=0.05),
        # a ragged batch with an odd width, as in a small model's tests
        dict(name="embed_grad_odd", op="embed_grad", vocab=50021, dim=1003, tokens=4099, grad="fp32", pads=0.1),
        # the dense gradient AdamW takes for the 163840 x 7168 embedding
        dict(name="embed_grad_batch", op="embed_grad", vocab=163840, dim=7168, tokens=16384, grad="bf16", pads=0.0),
        # scoring a few tokens: reads the head once
        dict(name="loss_16_tokens", op="loss", vocab=163840, dim=2048, tokens=16, dtype="bf16", ignored=0.0),
        # an evaluation batch over a vocabulary of odd size
        dict(name="loss_eval_batch", op="loss", vocab=50021, dim=2048, tokens=2048, dtype="fp16", ignored=0.1),
        # a short fine-tuning batch, a third of it prompt (ignored), odd in every size
        dict(name="loss_grad_odd", op="loss_grad", vocab=32003, dim=1000, tokens=999, dtype="bf16", ignored=0.33),
        # a pre-training micro-batch on the 163840 x 7168 head
        dict(name="loss_grad_batch", op="loss_grad", vocab=163840, dim=7168, tokens=4096, dtype="bf16", ignored=0.02),
        # a decoding batch spread over 40 of 128 experts: reads their weights once
        dict(name="experts_decode", op="experts", experts=128, active=40, tokens=64, width=2048, out=1408, dtype="bf16"),
        # the gate product of a training batch over 64 experts, three of them without a token
        dict(name="experts_batch", op="experts", experts=64, active=61, tokens=32768, width=2048, out=1408, dtype="bf16"),
        # both gradients of the down product of that batch
        dict(name="experts_grad_batch", op="experts_grad", experts=64, active=61, tokens=32768, width=1408, out=2048,
             dtype="bf16"),
        # a small fp16 run, odd in every size
        dict(name="experts_grad_odd", op="experts_grad", experts=7, active=6, tokens=3001, width=520, out=1000, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "embed_grad", "loss", "loss_grad", "experts", "experts_grad"])
    if op == "lookup":
        c = dict(op=op, vocab=_log(rng, 1000, 163840), dim=_log(rng, 64, 7168), tokens=_log(rng, 1, 32768),
                 table=rng.choice(["bf16", "fp16", "fp32"]), pads=rng.choice([0.0, 0.05]))
        c["out"] = rng.choice(["fp32", "bf16"]) if c["table"] == "fp32" else c["table"]
        return c
    if op == "embed_grad":
        return dict(op=op, vocab=_log(rng, 1000, 163840), dim=_log(rng, 64, 7168), tokens=_log(rng, 1, 16384),
                    grad=rng.choice(["bf16", "fp16", "fp32"]), pads=rng.choice([0.0, 0.1]))
    if op in ("loss", "loss_grad"):
        return dict(op=op, vocab=_log(rng, 1000, 163840), dim=8 * _log(rng, 16, 512), tokens=_log(rng, 1, 4096),
                    dtype=rng.choice(["bf16", "fp16"]), ignored=rng.choice([0.0, 0.3]))
    experts = _log(rng, 2, 128)
    return dict(op=op, experts=experts, active=rng.randint(max(1, experts // 3), experts), tokens=_log(rng, experts, 32768),
                width=8 * _log(rng, 16, 256), out=8 * _log(rng, 16, 256), dtype=rng.choice(["bf16", "fp16"]))


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _normal(gen, shape, std, dtype):
    x = torch.empty(shape, dtype=dtype, device=DEV)
    return x.normal_(0.0, std, generator=gen)


def _token_ids(gen, n, vocab):
    """Zipf-like token ids: rank r with probability ~ 1 / r, ranks spread over the vocabulary."""
    u = torch.rand(n, generator=gen, device=DEV, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab)) - 1.0).long().clamp_(0, vocab - 1)
    return rank * 7919 % vocab if vocab % 7919 else rank


def _sizes(case, seed):
    """Rows of each expert: `active` experts drawn at random share the tokens unevenly, the others have none."""
    rs = np.random.RandomState(seed % (1 << 31))
    chosen = rs.choice(case["experts"], case["active"], replace=False)
    active = min(case["active"], case["tokens"])
    rest = rs.multinomial(case["tokens"] - active, rs.dirichlet(np.full(active, 1.5)))
    sizes = np.zeros(case["experts"], dtype=np.int64)
    sizes[chosen[:active]] = 1 + rest
    return [int(s) for s in sizes]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1000003 * (seed + 1) % (1 << 62))
    op = case["op"]
    s = dict(case)
    if op in ("lookup", "embed_grad"):
        ids = _token_ids(gen, case["tokens"], case["vocab"])
        pad = case["vocab"] - 1
        mask = torch.rand(case["tokens"], generator=gen, device=DEV) < case["pads"]
        s["ids"] = torch.where(mask, torch.full_like(ids, pad), ids)
        s["pad"] = pad if case["pads"] else None
        s["scale"] = math.sqrt(case["dim"])
        if op == "lookup":
            s["weight"] = _normal(gen, (case["vocab"], case["dim"]), 0.02, DTYPES[case["table"]])
        else:
            s["dy"] = _normal(gen, (case["tokens"], case["dim"]), 1e-3, DTYPES[case["grad"]])
        return s
    dt = DTYPES[case["dtype"]]
    if op in ("loss", "loss_grad"):
        v, d, n = case["vocab"], case["dim"], case["tokens"]
        s["weight"] = _normal(gen, (v, d), 0.02, dt)
        t = _token_ids(gen, n, v)
        # hidden states that lean towards their target's row, some much, some hardly: losses from near 0 to above ln V
        lean = torch.rand(n, 1, generator=gen, device=DEV) * (18.0 / (4e-4 * d))
        s["hidden"] = (_normal(gen, (n, d), 1.0, torch.float32) + lean * s["weight"][t].float()).to(dt)
        skip = torch.rand(n, generator=gen, device=DEV) < case["ignored"]
        s["targets"] = torch.where(skip, torch.full_like(t, IGNORE), t)
        # the mean over the counted tokens
        s["row_scale"] = ((~skip).float() / (~skip).float().sum().clamp(min=1.0))
        return s
    sizes = _sizes(case, seed)
    s["sizes"] = sizes
    s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)
    s["x"] = _normal(gen, (case["tokens"], case["width"]), 1.0, dt)
    s["weight"] = _normal(gen, (case["experts"], case["out"], case["width"]), 0.02, dt)
    if op == "experts_grad":
        s["dy"] = _normal(gen, (case["tokens"], case["out"]), 0.05, dt)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def _plain(s):
    op = s["op"]
    if op == "lookup":
        y = s["weight"][s["ids"]].float() * s["scale"]
        if s["pad"] is not None:
            y = torch.where((s["ids"] == s["pad"])[:, None], torch.zeros_like(y), y)
        return {"y": y.to(DTYPES[s["out"]])}
    if op == "embed_grad":
        dy = s["dy"].float() * s["scale"]
        if s["pad"] is not None:
            dy = torch.where((s["ids"] == s["pad"])[:, None], torch.zeros_like(dy), dy)
        dw = torch.zeros((s["vocab"], s["dim"]), dtype=torch.float32, device=DEV)
        return {"d_table": dw.index_add_(0, s["ids"], dy)}
    if op in ("loss", "loss_grad"):
        h, w, t = s["hidden"].float(), s["weight"].float(), s["targets"]
        z = h @ w.t()
        top = z.max(dim=1, keepdim=True).values
        e = torch.exp(z - top)
        total = e.sum(dim=1, keepdim=True)
        lse = (top + torch.log(total))[:, 0]
        counted = t != IGNORE
        at = torch.where(counted, t, torch.zeros_like(t))
        rows = torch.arange(t.numel(), device=DEV)
        loss = torch.where(counted, lse - z[rows, at], torch.zeros_like(lse))
        if op == "loss":
            return {"loss": loss, "lse": lse}
        dz = e / total
        dz[rows, at] -= 1.0
        dz = dz * torch.where(counted, s["row_scale"], torch.zeros_like(s["row_scale"]))[:, None]
        return {"loss": loss, "lse": lse, "d_hidden": (dz @ w).to(s["hidden"].dtype),
                "d_weight": (dz.t() @ h).to(s["weight"].dtype)}
    dt = s["x"].dtype
    x, w = s["x"].float().split(s["sizes"]), s["weight"].float()
    if op == "experts":
        return {"y": torch.cat([a @ b.t() for a, b in zip(x, w)]).to(dt)}
    dy = s["dy"].float().split(s["sizes"])
    return {"d_x": torch.cat([a @ b for a, b in zip(dy, w)]).to(dt),
            "d_weight": torch.stack([a.t() @ b for a, b in zip(dy, x)]).to(dt)}


def _own(s):
    import optimizer_muon_step_gb300 as m
    op = s["op"]
    if op == "lookup":
        return {"y": m.muon_embedding_lookup(s["weight"], s["ids"], scale=s["scale"], padding_idx=s["pad"],
                                             out_dtype=DTYPES[s["out"]])}
    if op == "embed_grad":
        return {"d_table": m.muon_embedding_grad(s["dy"], s["ids"], s["vocab"], scale=s["scale"], padding_idx=s["pad"])}
    if op == "loss":
        loss, lse = m.muon_linear_ce(s["hidden"], s["weight"], s["targets"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    if op == "loss_grad":
        loss, lse, dh, dw = m.muon_linear_ce_grad(s["hidden"], s["weight"], s["targets"], row_scale=s["row_scale"],
                                                  ignore_index=IGNORE)
        return {"loss": loss, "lse": lse, "d_hidden": dh, "d_weight": dw}
    if op == "experts":
        return {"y": m.muon_expert_matmul(s["x"], s["weight"], s["offsets"])}
    return {"d_x": m.muon_expert_matmul(s["dy"], s["weight"], s["offsets"], transpose=True),
            "d_weight": m.muon_expert_wgrad(s["dy"], s["x"], s["offsets"])}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# What a pass cannot do without, and what it should give
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "lookup":
        n = case["tokens"] * case["dim"]
        return {"bytes": n * (BYTES[case["table"]] + BYTES[case["out"]]) + 8 * case["tokens"], "flops": n}
    if op == "embed_grad":
        n = case["tokens"] * case["dim"]
        return {"bytes": n * BYTES[case["grad"]] + 8 * case["tokens"] + 4 * case["vocab"] * case["dim"], "flops": 2 * n}
    if op in ("loss", "loss_grad"):
        v, d, n = case["vocab"], case["dim"], case["tokens"]
        once = 2 * (v * d + n * d) + 8 * n + 8 * n
        if op == "loss":
            return {"bytes": once, "flops": 2 * n * v * d}
        return {"bytes": once + 4 * n + 2 * (v * d + n * d), "flops": 6 * n * v * d}
    active = min(case["active"], case["tokens"])
    n, k, o = case["tokens"], case["width"], case["out"]
    if op == "experts":
        return {"bytes": 2 * (n * k + active * k * o + n * o) + 4 * (case["experts"] + 1), "flops": 2 * n * k * o}
    return {"bytes": 2 * (2 * n * k + n * o + active * k * o + case["experts"] * k * o) + 4 * (case["experts"] + 1),
            "flops": 4 * n * k * o}


def exact(case, seed):
    """The definitions, row block by row block, in fp64."""
    op = case["op"]
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    if op == "lookup":
        y = s["weight"].index_select(0, s["ids"]).double().mul_(float(np.float32(s["scale"])))
        if s["pad"] is not None:
            y[s["ids"].eq(s["pad"])] = 0.0
        return {"y": y}
    if op == "embed_grad":
        live = torch.ones_like(s["ids"], dtype=torch.bool) if s["pad"] is None else s["ids"].ne(s["pad"])
        g = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device=DEV)
        g.index_put_((s["ids"][live],), s["dy"][live].double() * float(np.float32(s["scale"])), accumulate=True)
        return {"d_table": g}
    if op in ("loss", "loss_grad"):
        n, w = case["tokens"], s["weight"].double()
        loss, lse, dh = [], [], []
        dw = torch.zeros_like(w) if op == "loss_grad" else None
        for b in range(0, n, 512):
            h, t = s["hidden"][b:b + 512].double(), s["targets"][b:b + 512]
            z = torch.einsum("nd,vd->nv", h, w)
            norm = torch.logsumexp(z, 1)
            lse.append(norm)
            hot = torch.zeros_like(z)
            live = t.ge(0)
            hot[live.nonzero()[:, 0], t[live]] = 1.0
            loss.append(torch.where(live, norm - (z * hot).sum(1), 0.0))
            if dw is not None:
                q = (torch.exp(z - norm[:, None]) - hot) * (s["row_scale"][b:b + 512].double() * live)[:, None]
                dh.append(torch.einsum("nv,vd->nd", q, w))
                dw += torch.einsum("nv,nd->vd", q, h)
        got = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
        if dw is not None:
            got["d_hidden"], got["d_weight"] = torch.cat(dh), dw
        return got
    n, e = case["tokens"], case["experts"]
    a = s["x"] if op == "experts" else s["dy"]
    rows = torch.zeros(n, case["out"] if op == "experts" else case["width"], dtype=torch.float64, device=DEV)
    dw = None if op == "experts" else torch.zeros(e, case["out"], case["width"], dtype=torch.float64, device=DEV)
    first = 0
    for i, size in enumerate(s["sizes"]):
        part = slice(first, first + size)
        w = s["weight"][i].double()
        rows[part] = a[part].double() @ (w.T if op == "experts" else w)
        if dw is not None and size:
            dw[i] = torch.einsum("no,nk->ok", s["dy"][part].double(), s["x"][part].double())
        first += size
    return {"y": rows} if dw is None else {"d_x": rows, "d_weight": dw}
