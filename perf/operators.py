"""Cases for timing the operators at the ends of a training step.

The optimizer step reads gradients that three operators around it write:

* the embedding lookup with scaling, and its gradient by sorted tokens
  (``embed_forward``, ``embed_backward``);
* the softmax cross entropy of a linear head over a large vocabulary, in
  pieces of the vocabulary, and its gradient (``lm_loss_forward``,
  ``lm_loss_backward``);
* matrix products grouped by expert with ragged sizes, and the expert
  weights' gradient (``expert_matmul``, ``expert_wgrad``).

``run`` computes a case in elementary torch operations, in fp32, rounded
once; with ``own`` set it makes the framework's calls instead.  ``exact``
gives the same outputs from the definitions in fp64.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
IGNORED = -100          # target of a position that has no label
PAD = -1                # id of a padding position


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 16 sequences: latency only
        dict(name="lookup_decode_16", op="embed_fwd", n=16, vocab=32000, dim=2048,
             dtype="bf16", pad=0.0),
        # the token embedding of a packed training batch, largest vocabulary
        dict(name="lookup_train_32k_large", op="embed_fwd", n=32768, vocab=163840, dim=7168,
             dtype="bf16", pad=0.0),
        # gradient of a small fine-tuning batch with padding, fp32 gradients, odd width
        dict(name="lookup_grad_ragged_fp32", op="embed_bwd", n=4099, vocab=33001, dim=1001,
             dtype="fp32", pad=0.2),
        # gradient of one micro-batch, the dense workload's embedding
        dict(name="lookup_grad_8k", op="embed_bwd", n=8191, vocab=32000, dim=2048,
             dtype="bf16", pad=0.05),
        # gradient of a packed training batch, largest vocabulary
        dict(name="lookup_grad_32k_large", op="embed_bwd", n=32768, vocab=163840, dim=7168,
             dtype="bf16", pad=0.0),
        # scoring a short answer: forward only, few rows
        dict(name="loss_score_33", op="loss_fwd", n=33, vocab=32000, dim=2048, dtype="bf16",
             ignored=0.0),
        # a fine-tuning step in fp32 on odd sizes
        dict(name="loss_step_ragged_fp32", op="loss_step", n=515, vocab=33001, dim=500,
             dtype="fp32", ignored=0.3),
        # a training micro-batch of the dense workload's LM head
        dict(name="loss_step_8k", op="loss_step", n=8192, vocab=32000, dim=2048, dtype="bf16",
             ignored=0.05),
        # a training micro-batch at the largest vocabulary and width
        dict(name="loss_step_4k_large", op="loss_step", n=4096, vocab=163840, dim=7168,
             dtype="bf16", ignored=0.05),
        # decoding: 8 routed rows over 64 experts, bound by the weights read
        dict(name="experts_decode_8", op="experts_fwd", rows=8, experts=64, k=2048, n=1408,
             dtype="bf16", trans=False, empty=0.0),
        # off-grid expert shapes, few rows each, weights stored [out, in]
        dict(name="experts_step_odd", op="experts_step", rows=1777, experts=13, k=1001, n=703,
             dtype="bf16", trans=True, empty=0.3),
        # a training micro-batch over 128 experts of the largest shape
        dict(name="experts_step_64k_large", op="experts_step", rows=65536, experts=128, k=7168,
             n=2048, dtype="bf16", trans=False, empty=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature width: usually a multiple of 64, sometimes odd."""
    d = _log_int(rng, lo, hi)
    return d if rng.random() < 0.2 else max(64, d // 64 * 64)


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "loss_fwd", "loss_step", "experts_fwd",
                     "experts_step"])
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    if op.startswith("embed"):
        return dict(op=op, n=_log_int(rng, 16, 32768), vocab=_log_int(rng, 8192, 163840),
                    dim=_width(rng, 256, 7168), dtype=dtype, pad=rng.choice([0.0, 0.1, 0.4]))
    if op.startswith("loss"):
        c = dict(op=op, n=_log_int(rng, 16, 8192), vocab=_log_int(rng, 8192, 163840),
                 dim=_width(rng, 256, 7168), dtype=dtype, ignored=rng.choice([0.0, 0.1, 0.5]))
        top = 4096 * 163840 * 7168 // (8 if dtype == "fp32" else 1)
        while c["n"] * c["vocab"] * c["dim"] > top:
            c["n"] = c["n"] * 2 // 3
        return c
    c = dict(op=op, rows=_log_int(rng, 8, 65536), experts=_log_int(rng, 4, 128),
             k=_width(rng, 256, 7168), n=_width(rng, 256, 4096), dtype=dtype,
             trans=rng.random() < 0.5, empty=rng.choice([0.0, 0.1, 0.5]))
    top = 128 * 7168 * 2048 // (2 if dtype == "fp32" else 1)
    while c["experts"] * c["k"] * c["n"] > top:
        c["experts"] = c["experts"] * 2 // 3
    top = 65536 * 7168 * 2048 // (8 if dtype == "fp32" else 1)
    while c["rows"] * c["k"] * c["n"] > top:
        c["rows"] = c["rows"] * 2 // 3
    return c


# ------------------------------------------------------------------ inputs

def _tokens(g, n, vocab, missing, marker):
    """Token ids as a text has them: frequencies fall with the rank, ranks
    are spread over the vocabulary; a share of positions has none."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab + 1.0)).floor().long() - 1
    ids = (rank.clamp_(0, vocab - 1) * 7919 + 13) % vocab
    if missing:
        gone = torch.rand(n, generator=g, device="cuda") < missing
        ids = torch.where(gone, torch.full_like(ids, marker), ids)
    return ids


def _normal(g, shape, std, dtype):
    return torch.empty(shape, device="cuda", dtype=DTYPES[dtype]).normal_(0.0, std, generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, dt = case["op"], case["dtype"]
    s = {"case": case}
    if op.startswith("embed"):
        n, vocab, dim = case["n"], case["vocab"], case["dim"]
        s["ids"] = _tokens(g, n, vocab, case["pad"], PAD)
        s["scale"] = math.sqrt(dim)
        if op == "embed_fwd":
            s["table"] = _normal(g, (vocab, dim), 0.02, dt)
            s["out"] = torch.empty(n, dim, device="cuda", dtype=DTYPES[dt])
        else:
            s["dout"] = _normal(g, (n, dim), 1e-3, dt)
            s["dtable"] = torch.empty(vocab, dim, device="cuda", dtype=DTYPES[dt])
    elif op.startswith("loss"):
        n, vocab, dim = case["n"], case["vocab"], case["dim"]
        s["hidden"] = _normal(g, (n, dim), 1.0, dt)
        s["weight"] = _normal(g, (vocab, dim), 0.02, dt)
        s["targets"] = _tokens(g, n, vocab, case["ignored"], IGNORED)
        # the gradient of the mean over the labelled positions
        labelled = int((s["targets"] >= 0).sum())
        s["dloss"] = torch.full((n,), 1.0 / max(1, labelled), device="cuda")
        if op == "loss_step":
            s["dhidden"] = torch.empty_like(s["hidden"])
            s["dweight"] = torch.empty_like(s["weight"])
    else:
        rows, experts, k, n = case["rows"], case["experts"], case["k"], case["n"]
        host = np.random.Generator(np.random.PCG64(int(seed)))
        # a router's load: uneven, some experts without a row
        share = np.exp(host.normal(0.0, 0.4, experts))
        share[host.random(experts) < case["empty"]] = 0.0
        if share.sum() == 0.0:
            share[0] = 1.0
        counts = host.multinomial(rows, share / share.sum())
        s["counts"] = [int(c) for c in counts]
        s["offsets"] = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32,
                                    device="cuda")
        s["x"] = _normal(g, (rows, k), 1.0, dt)
        s["w"] = _normal(g, (experts, n, k) if case["trans"] else (experts, k, n), 0.02, dt)
        s["y"] = torch.empty(rows, n, device="cuda", dtype=DTYPES[dt])
        if op == "experts_step":
            s["dy"] = _normal(g, (rows, n), 1e-2, dt)
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty_like(s["w"])
    if own:
        import muon_newton_schulz_amd as M
        if op == "embed_bwd":
            s["ws"] = torch.empty(M.embed_backward_workspace_size(n, vocab, dim),
                                  dtype=torch.uint8, device="cuda")
        elif op.startswith("loss"):
            s["ws"] = torch.empty(M.lm_loss_workspace_size(n, vocab, dim, dt,
                                                           backward=op == "loss_step"),
                                  dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ passes

def _run_own(s):
    import muon_newton_schulz_amd as M
    op = s["case"]["op"]
    if op == "embed_fwd":
        return M.embed_forward(s["table"], s["ids"], s["scale"], out=s["out"])
    if op == "embed_bwd":
        return M.embed_backward(s["dout"], s["ids"], s["dtable"], s["scale"], workspace=s["ws"])
    if op == "loss_fwd":
        return M.lm_loss_forward(s["hidden"], s["weight"], s["targets"], workspace=s["ws"])
    if op == "loss_step":
        loss, lse = M.lm_loss_forward(s["hidden"], s["weight"], s["targets"], workspace=s["ws"])
        dh, dw = M.lm_loss_backward(s["hidden"], s["weight"], s["targets"], lse, s["dloss"],
                                    dhidden=s["dhidden"], dweight=s["dweight"],
                                    workspace=s["ws"])
        return loss, lse, dh, dw
    trans = s["case"]["trans"]
    y = M.expert_matmul(s["x"], s["w"], s["offsets"], trans=trans, out=s["y"])
    if op == "experts_fwd":
        return y
    dx = M.expert_matmul(s["dy"], s["w"], s["offsets"], trans=not trans, out=s["dx"])
    a, b = (s["dy"], s["x"]) if trans else (s["x"], s["dy"])
    return y, dx, M.expert_wgrad(a, b, s["offsets"], s["dw"])


def _plain_embed(s):
    ids, dt = s["ids"], DTYPES[s["case"]["dtype"]]
    present = ids >= 0
    safe = ids.clamp(min=0)
    if s["case"]["op"] == "embed_fwd":
        rows = s["table"][safe].float() * s["scale"]
        return torch.where(present[:, None], rows, torch.zeros_like(rows)).to(dt)
    acc = torch.zeros(s["case"]["vocab"], s["case"]["dim"], device="cuda")
    rows = s["dout"].float() * present[:, None]
    acc.index_add_(0, safe, rows)
    return (acc * s["scale"]).to(dt)


def _plain_loss(s):
    h, w = s["hidden"].float(), s["weight"].float()
    t = s["targets"]
    labelled, safe = t >= 0, t.clamp(min=0)
    logits = h @ w.t()
    top = logits.max(dim=1).values
    lse = top + (logits - top[:, None]).exp().sum(dim=1).log()
    at = logits.gather(1, safe[:, None])[:, 0]
    loss = torch.where(labelled, lse - at, torch.zeros_like(lse))
    if s["case"]["op"] == "loss_fwd":
        return loss, lse
    g = (logits - lse[:, None]).exp()
    g[torch.arange(t.numel(), device="cuda"), safe] -= 1.0
    g *= (s["dloss"] * labelled)[:, None]
    dt = DTYPES[s["case"]["dtype"]]
    return loss, lse, (g @ w).to(dt), (g.t() @ h).to(dt)


def _plain_experts(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    step = case["op"] == "experts_step"
    x = s["x"].float()
    y = torch.empty(case["rows"], case["n"], device="cuda")
    if step:
        dy = s["dy"].float()
        dx = torch.empty(case["rows"], case["k"], device="cuda")
        dw = torch.zeros(s["w"].shape, device="cuda", dtype=dt)
    r = 0
    for e, c in enumerate(s["counts"]):
        if c:
            we = s["w"][e].float()
            if case["trans"]:
                we = we.t()
            y[r:r + c] = x[r:r + c] @ we
            if step:
                dx[r:r + c] = dy[r:r + c] @ we.t()
                a, b = (dy, x) if case["trans"] else (x, dy)
                dw[e] = (a[r:r + c].t() @ b[r:r + c]).to(dt)
        r += c
    if not step:
        return y.to(dt)
    return y.to(dt), dx.to(dt), dw


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op.startswith("embed"):
        return _plain_embed(state)
    if op.startswith("loss"):
        return _plain_loss(state)
    return _plain_experts(state)


# -------------------------------------------------------------------- work

def work(case):
    """Bytes and operations of one pass: every input read once, every output
    written once, multiply and add counted as two.  A lookup reads the rows
    that its positions name, an expert's weights count only if rows can
    reach it; the loss step's product of the logits counts once."""
    sz, op = SIZE[case["dtype"]], case["op"]
    if op.startswith("embed"):
        n, vocab, dim = case["n"], case["vocab"], case["dim"]
        if op == "embed_fwd":
            # ranks are log-uniform: the expected number of distinct rows
            rank = np.arange(1, vocab + 1, dtype=np.float64)
            p = np.log1p(1.0 / rank) / math.log(vocab + 1.0)
            distinct = float((-np.expm1(n * np.log1p(-p))).sum())
            return {"bytes": distinct * dim * sz + n * dim * sz + 8 * n, "flops": n * dim}
        return {"bytes": n * dim * sz + vocab * dim * sz + 8 * n, "flops": n * dim}
    if op.startswith("loss"):
        n, vocab, dim = case["n"], case["vocab"], case["dim"]
        fwd = 2 * n * vocab * dim
        read = (n + vocab) * dim * sz + 8 * n
        if op == "loss_fwd":
            return {"bytes": read + 8 * n, "flops": fwd}
        return {"bytes": 2 * read + 12 * n, "flops": 3 * fwd}
    rows, experts, k, n = case["rows"], case["experts"], case["k"], case["n"]
    reached = min(experts * (1.0 - case["empty"]), rows)
    fwd = 2 * rows * k * n
    if op == "experts_fwd":
        return {"bytes": (reached * k * n + rows * (k + n)) * sz, "flops": fwd}
    return {"bytes": ((reached + experts) * k * n + 2 * rows * (k + n)) * sz, "flops": 3 * fwd}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        out = torch.zeros(case["n"], case["dim"], dtype=torch.float64, device="cuda")
        at = (s["ids"] >= 0).nonzero()[:, 0]
        out[at] = s["table"].index_select(0, s["ids"][at]).double() * s["scale"]
        return out
    if op == "embed_bwd":
        out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
        at = (s["ids"] >= 0).nonzero()[:, 0]
        return out.index_add_(0, s["ids"][at], s["dout"][at].double() * s["scale"])
    if op.startswith("loss"):
        n = case["n"]
        w = s["weight"].double()
        loss = torch.zeros(n, dtype=torch.float64, device="cuda")
        lse = torch.empty_like(loss)
        step = op == "loss_step"
        if step:
            dh = torch.empty(n, case["dim"], dtype=torch.float64, device="cuda")
            dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
        for r0 in range(0, n, 1024):
            r1 = min(n, r0 + 1024)
            h = s["hidden"][r0:r1].double()
            logits = torch.mm(h, w.t())
            lse[r0:r1] = torch.logsumexp(logits, 1)
            t = s["targets"][r0:r1]
            at = (t >= 0).nonzero()[:, 0]
            loss[r0 + at] = lse[r0 + at] - logits[at, t[at]]
            if step:
                g = torch.softmax(logits, 1)
                g[at, t[at]] -= 1.0
                scale = torch.zeros(r1 - r0, dtype=torch.float64, device="cuda")
                scale[at] = s["dloss"][r0:r1].double()[at]
                g.mul_(scale.unsqueeze(1))
                dh[r0:r1] = torch.mm(g, w)
                dw.addmm_(g.t(), h)
        return (loss, lse, dh, dw) if step else (loss, lse)
    bounds = s["offsets"].tolist()
    step = op == "experts_step"
    y = torch.empty(case["rows"], case["n"], dtype=torch.float64, device="cuda")
    if step:
        dx = torch.empty(case["rows"], case["k"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        w = s["w"][e].double()
        x = s["x"][lo:hi].double()
        y[lo:hi] = torch.mm(x, w.t() if case["trans"] else w)
        if step:
            d = s["dy"][lo:hi].double()
            dx[lo:hi] = torch.mm(d, w if case["trans"] else w.t())
            dw[e] = torch.mm(d.t(), x) if case["trans"] else torch.mm(x.t(), d)
    return (y, dx, dw) if step else y
