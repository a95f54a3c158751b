"""Cases for timing the losses of fine-tuning behind a language-model head.

Cross entropy teaches the next token of a text.  Three more losses consume
what the same head computes:

* distillation from a teacher's top logits, through the linear head, without
  storing the student's logits (``distill_loss_forward``,
  ``distill_loss_backward``);
* the clipped policy loss with a KL term over packed sequences
  (``policy_loss_forward``, ``policy_loss_backward``), from the token losses
  that ``lm_loss_forward`` returns; its gradient is the ``dloss`` that
  ``lm_loss_backward`` takes;
* the preference loss over pairs of packed sequences
  (``preference_loss_forward``, ``preference_loss_backward``), with the same
  inputs and gradient.

``run`` computes a case in elementary torch operations, in fp32 (the losses
over sequences in fp64: ratios next to a clip border, long sums), rounded
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
ABSENT = -1             # id of a missing entry of a teacher's list


# ------------------------------------------------------------------- cases

def listed():
    return [
        # evaluating a student on a short text: forward only, few rows
        dict(name="distill_score_33", op="distill_fwd", n=33, vocab=32000, dim=2048, top=32,
             dtype="bf16", teacher="fp32", temperature=1.0, absent=0.0),
        # a fine-tuning step in fp32 on odd sizes, lists with gaps, softened
        dict(name="distill_step_ragged_fp32", op="distill_step", n=515, vocab=33001, dim=500,
             top=17, dtype="fp32", teacher="fp32", temperature=2.0, absent=0.3),
        # a training micro-batch of the dense workload's head
        dict(name="distill_step_8k", op="distill_step", n=8192, vocab=32000, dim=2048, top=64,
             dtype="bf16", teacher="bf16", temperature=1.0, absent=0.05),
        # a training micro-batch at the largest vocabulary and width
        dict(name="distill_step_4k_large", op="distill_step", n=4096, vocab=163840, dim=7168,
             top=128, dtype="bf16", teacher="fp32", temperature=2.0, absent=0.0),
        # one update on 16 short answers: latency only
        dict(name="policy_step_16", op="policy_step", n=2000, sequences=16, tail=48, prompt=0.3,
             ref=True, per_token=False, empty=0.0, mean=True),
        # watching the KL and the clipped share of a batch: forward only, no mask
        dict(name="policy_watch_64k", op="policy_fwd", n=65536, sequences=64, tail=0, prompt=0.0,
             ref=True, per_token=False, empty=0.0, mean=True),
        # a few very long trajectories, an advantage for each token, no reference
        dict(name="policy_step_long", op="policy_step", n=1000003, sequences=5, tail=0,
             prompt=0.1, ref=False, per_token=True, empty=0.0, mean=False),
        # the largest batch: 512 prompts with 16 answers of about 4000 tokens each
        dict(name="policy_step_8192", op="policy_step", n=33554432, sequences=8192, tail=4096,
             prompt=0.2, ref=True, per_token=False, empty=0.02, mean=True),
        # a few pairs of short answers: latency only
        dict(name="preference_step_8", op="preference_step", n=3001, sequences=16, tail=63,
             prompt=0.5, ref=True, empty=0.0, mean=False, kind="logistic", smoothing=0.0),
        # scoring a held-out set, mean rewards without a reference
        dict(name="preference_score_1k", op="preference_fwd", n=524288, sequences=2048, tail=0,
             prompt=0.3, ref=False, empty=0.0, mean=True, kind="logistic", smoothing=0.0),
        # the largest batch of pairs, some with an answer that was cut away
        dict(name="preference_step_4k", op="preference_step", n=16777213, sequences=8192, tail=0,
             prompt=0.4, ref=True, empty=0.02, mean=False, kind="logistic", smoothing=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature width: usually a multiple of 64, sometimes odd."""
    d = _log_int(rng, lo, hi)
    return d if rng.random() < 0.2 else max(64, d // 64 * 64)


def draw(rng):
    op = rng.choice(["distill_fwd", "distill_step", "policy_fwd", "policy_step",
                     "preference_fwd", "preference_step"])
    if op.startswith("distill"):
        dtype = "fp32" if rng.random() < 0.2 else "bf16"
        c = dict(op=op, n=_log_int(rng, 16, 8192), vocab=_log_int(rng, 8192, 163840),
                 dim=_width(rng, 256, 7168), top=_log_int(rng, 1, 256), dtype=dtype,
                 teacher=rng.choice(["bf16", "fp32"]), temperature=rng.choice([1.0, 2.0, 0.7]),
                 absent=rng.choice([0.0, 0.1, 0.5]))
        top = 4096 * 163840 * 7168 // (8 if dtype == "fp32" else 1)
        while c["n"] * c["vocab"] * c["dim"] > top:
            c["n"] = c["n"] * 2 // 3
        return c
    n = _log_int(rng, 256, 33554432 if op.startswith("policy") else 16777216)
    c = dict(op=op, n=n, sequences=2 * _log_int(rng, 1, max(1, min(8192, n // 32))),
             tail=rng.choice([0, 0, 17, n // 20]), prompt=rng.choice([0.0, 0.2, 0.6]),
             ref=rng.random() < 0.7, empty=rng.choice([0.0, 0.1]), mean=rng.random() < 0.5)
    if op.startswith("policy"):
        return dict(c, per_token=rng.random() < 0.4)
    return dict(c, kind=rng.choice(["logistic", "hinge", "squared"]),
                smoothing=rng.choice([0.0, 0.1]))


# the settings that a run fixes once
CLIP_LOW, CLIP_HIGH, KL_WEIGHT = 0.2, 0.28, 0.05
BETA = {False: 0.1, True: 2.0}      # by mean: of a sum of ratios, of their mean
MARGIN = {False: 0.0, True: 0.5}


# ------------------------------------------------------------------ inputs

def _normal(g, shape, std, dtype):
    return torch.empty(shape, device="cuda", dtype=DTYPES[dtype]).normal_(0.0, std, generator=g)


def _top_ids(g, n, top, vocab, absent):
    """Each row's list: tokens of all ranks (their logarithms spread evenly),
    ranks spread over the vocabulary, a share of the entries missing."""
    u = torch.rand(n, top, generator=g, device="cuda", dtype=torch.float64)
    k = torch.arange(top, device="cuda", dtype=torch.float64)
    rank = torch.exp((k + u) / top * math.log(vocab)).floor().long() - 1
    ids = ((rank + torch.arange(top, device="cuda")) * 7919 + 13) % vocab
    if absent:
        gone = torch.rand(n, top, generator=g, device="cuda") < absent
        ids = torch.where(gone, torch.full_like(ids, ABSENT), ids)
    return ids


def _sequences(g, case, seed, s):
    """Packed sequences of uneven lengths, some empty, their prompts masked."""
    n, count, tail = case["n"], case["sequences"], case["tail"]
    host = np.random.Generator(np.random.PCG64(int(seed)))
    share = np.exp(host.normal(0.0, 0.5, count))
    share[host.random(count) < case["empty"]] = 0.0
    if share.sum() == 0.0:
        share[0] = 1.0
    lengths = host.multinomial(n - tail, share / share.sum())
    s["offsets"] = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")
    if case["prompt"]:
        length = torch.tensor(lengths, device="cuda")
        answer = (length * 2 * case["prompt"]
                  * torch.rand(count, generator=g, device="cuda")).long().clamp(max=length)
        first = torch.repeat_interleave(s["offsets"][:-1] + answer, length)
        mask = torch.arange(n - tail, device="cuda") >= first
        s["mask"] = torch.cat([mask, torch.zeros(tail, dtype=torch.bool, device="cuda")])
    else:
        s["mask"] = None
    # token losses: mostly small, some large
    s["nll"] = torch.rand(n, generator=g, device="cuda").clamp_(min=1e-6).log_().neg_().square_()
    s["ref"] = None
    if case["ref"]:
        noise = torch.empty(n, device="cuda").normal_(0.0, 0.1, generator=g)
        s["ref"] = (s["nll"] + noise).clamp_(min=0.0)
    s["dnll"] = torch.zeros(n, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op.startswith("distill"):
        n, vocab, dim, dt = case["n"], case["vocab"], case["dim"], case["dtype"]
        s["hidden"] = _normal(g, (n, dim), 1.0, dt)
        s["weight"] = _normal(g, (vocab, dim), 0.02, dt)
        s["ids"] = _top_ids(g, n, case["top"], vocab, case["absent"])
        s["teacher"] = _normal(g, (n, case["top"]), 2.0, case["teacher"])
        # the gradient of the mean over the positions
        s["dloss"] = torch.full((n,), 1.0 / n, device="cuda")
        if op == "distill_step":
            s["dhidden"] = torch.empty_like(s["hidden"])
            s["dweight"] = torch.empty_like(s["weight"])
        return s
    _sequences(g, case, seed, s)
    if op.startswith("policy"):
        noise = torch.empty(case["n"], device="cuda").normal_(0.0, 0.15, generator=g)
        s["old"] = (s["nll"] + noise).clamp_(min=0.0)
        s["advantages"] = torch.randn(case["n"] if case["per_token"] else case["sequences"],
                                      generator=g, device="cuda")
        s["dloss"] = torch.full((case["sequences"],), 1.0 / case["sequences"], device="cuda")
    else:
        pairs = case["sequences"] // 2
        s["dloss"] = torch.full((pairs,), 1.0 / pairs, device="cuda")
    return s


# ------------------------------------------------------------------ passes

def _workspace(s, size):
    """What a program keeps from step to step: made at the first pass."""
    if "ws" not in s:
        s["ws"] = torch.empty(size(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    import muon_newton_schulz_amd as M
    case = s["case"]
    op = case["op"]
    step = op.endswith("step")
    if op.startswith("distill"):
        ws = _workspace(s, lambda: M.distill_loss_workspace_size(
            case["n"], case["vocab"], case["dim"], case["top"], case["dtype"], backward=step))
        t = case["temperature"]
        loss, lse, logp = M.distill_loss_forward(s["hidden"], s["weight"], s["ids"], s["teacher"],
                                                 temperature=t, workspace=ws)
        if not step:
            return loss, lse, logp
        dh, dw = M.distill_loss_backward(s["hidden"], s["weight"], s["ids"], s["teacher"], lse,
                                         logp, s["dloss"], temperature=t, dhidden=s["dhidden"],
                                         dweight=s["dweight"], workspace=ws)
        return loss, lse, logp, dh, dw
    ws = _workspace(s, lambda: M.sequence_loss_workspace_size(case["n"], case["sequences"]))
    if op.startswith("policy"):
        how = dict(ref_nll=s["ref"], mask=s["mask"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                   kl_weight=KL_WEIGHT if case["ref"] else 0.0, mean=case["mean"],
                   per_token=case["per_token"])
        loss, kl, count, clipped = M.policy_loss_forward(
            s["nll"], s["old"], s["advantages"], s["offsets"], workspace=ws, **how)
        if not step:
            return loss, kl, count, clipped
        dnll = M.policy_loss_backward(s["nll"], s["old"], s["advantages"], s["offsets"], count,
                                      s["dloss"], dnll=s["dnll"], **how)
        return loss, kl, count, clipped, dnll
    how = dict(mask=s["mask"], beta=BETA[case["mean"]], kind=case["kind"],
               smoothing=case["smoothing"] if case["kind"] == "logistic" else 0.0,
               mean=case["mean"])
    loss, margin, reward, count = M.preference_loss_forward(
        s["nll"], s["offsets"], ref_nll=s["ref"], margin=MARGIN[case["mean"]], workspace=ws, **how)
    if not step:
        return loss, margin, reward, count
    dnll = M.preference_loss_backward(s["offsets"], margin, count, s["dloss"], dnll=s["dnll"],
                                      **how)
    return loss, margin, reward, count, dnll


def _plain_distill(s):
    case = s["case"]
    h, w, ids = s["hidden"].float(), s["weight"].float(), s["ids"]
    there = (ids >= 0) & (ids < case["vocab"])
    safe = torch.where(there, ids, torch.zeros_like(ids))
    logits = (h @ w.t()) / case["temperature"]
    top = logits.max(dim=1, keepdim=True).values
    lse = top + (logits - top).exp().sum(dim=1, keepdim=True).log()
    logp = logits.gather(1, safe) - lse
    z = s["teacher"].float() / case["temperature"]
    z = torch.where(there, z, torch.full_like(z, -1e30))
    z = z - z.max(dim=1, keepdim=True).values
    e = torch.where(there, z.exp(), torch.zeros_like(z))
    total = e.sum(dim=1, keepdim=True)
    some = total > 0.0
    total = torch.where(some, total, torch.ones_like(total))
    q = e / total
    zero = torch.zeros_like(z)
    loss = torch.where(there, q * ((z - total.log()) - logp), zero).sum(dim=1)
    logp = torch.where(there, logp, zero)
    if case["op"] == "distill_fwd":
        return loss, lse[:, 0], logp
    g = (logits - lse).exp()
    g.scatter_add_(1, safe, -q)
    g *= (s["dloss"] / case["temperature"])[:, None] * some
    dt = DTYPES[case["dtype"]]
    return loss, lse[:, 0], logp, (g @ w).to(dt), (g.t() @ h).to(dt)


def _spans(s):
    """First and last positions of the sequences; each position's sequence and
    whether it counts."""
    off = s["offsets"].long()
    n = s["nll"].numel()
    seq = torch.searchsorted(off, torch.arange(n, device="cuda"), right=True) - 1
    counts = (seq >= 0) & (seq < off.numel() - 1)
    seq = seq.clamp(0, off.numel() - 2)
    if s["mask"] is not None:
        counts = counts & s["mask"]
    return off[:-1], off[1:], seq, counts


def _sums(values, lo, hi):
    c = torch.cat([values.new_zeros(1), values.cumsum(0)])
    return c[hi] - c[lo]


def _plain_policy(s):
    case = s["case"]
    lo, hi, seq, counts = _spans(s)
    nll = s["nll"].double()
    a = s["advantages"].double()
    if not case["per_token"]:
        a = a[seq]
    zero = torch.zeros_like(nll)
    r = (s["old"].double() - nll).exp()
    cut = ((a > 0) & (r > 1.0 + CLIP_HIGH)) | ((a < 0) & (r < 1.0 - CLIP_LOW))
    token = -torch.minimum(r * a, r.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * a)
    grad = torch.where(cut, zero, r * a)
    k = zero
    if case["ref"]:
        x = nll - s["ref"].double()
        k = x.expm1() - x
        token = token + KL_WEIGHT * k
        grad = grad + KL_WEIGHT * x.expm1()
    count = _sums(counts.long(), lo, hi)
    clipped = _sums((counts & cut).long(), lo, hi)
    part = torch.ones_like(count, dtype=torch.float64)
    if case["mean"]:
        part = 1.0 / count.clamp(min=1)
    loss = (_sums(torch.where(counts, token, zero), lo, hi) * part).float()
    kl = (_sums(torch.where(counts, k, zero), lo, hi) * part).float()
    out = loss, kl, count.int(), clipped.int()
    if case["op"] == "policy_fwd":
        return out
    each = (s["dloss"].double() * part)[seq]
    return *out, torch.where(counts, grad * each, zero).float()


def _plain_preference(s):
    case = s["case"]
    lo, hi, seq, counts = _spans(s)
    ratio = -s["nll"].double()
    if case["ref"]:
        ratio = ratio + s["ref"].double()
    zero = torch.zeros_like(ratio)
    count = _sums(counts.long(), lo, hi)
    scale = torch.full_like(count, BETA[case["mean"]], dtype=torch.float64)
    if case["mean"]:
        scale = scale / count.clamp(min=1)
    reward = _sums(torch.where(counts, ratio, zero), lo, hi) * scale
    x = reward[0::2] - reward[1::2] - MARGIN[case["mean"]]
    e = case["smoothing"]
    if case["kind"] == "logistic":
        soft = (-x.abs()).exp().log1p()
        loss = (1.0 - e) * (soft + (-x).clamp(min=0)) + e * (soft + x.clamp(min=0))
        slope = e - 1.0 / (1.0 + x.exp())
    elif case["kind"] == "hinge":
        loss, slope = (1.0 - x).clamp(min=0), -(x < 1.0).double()
    else:
        loss, slope = (1.0 - x) ** 2, 2.0 * (x - 1.0)
    both = (count[0::2] > 0) & (count[1::2] > 0)
    loss = torch.where(both, loss, torch.zeros_like(loss))
    out = loss.float(), x.float(), reward.float(), count.int()
    if case["op"] == "preference_fwd":
        return out
    d = torch.where(both, slope * s["dloss"].double(), torch.zeros_like(loss))
    each = torch.stack([-d, d], 1).reshape(-1) * scale
    return *out, torch.where(counts, each[seq], zero).float()


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op.startswith("distill"):
        return _plain_distill(state)
    if op.startswith("policy"):
        return _plain_policy(state)
    return _plain_preference(state)


# -------------------------------------------------------------------- work

def work(case):
    """Bytes and operations of one pass: every input read once, every output
    written once, multiply and add counted as two; a distillation step's
    product of the logits counts once.  A token of the losses over sequences
    takes about 20 operations forward and as many backward."""
    op = case["op"]
    step = op.endswith("step")
    if op.startswith("distill"):
        sz, n, vocab, dim, top = (SIZE[case["dtype"]], case["n"], case["vocab"], case["dim"],
                                  case["top"])
        rows = (n + vocab) * dim * sz
        lists = n * top * (8 + SIZE[case["teacher"]] + 4)
        fwd = 2 * n * vocab * dim
        if step:
            return {"bytes": 2 * rows + lists + 12 * n, "flops": 3 * fwd}
        return {"bytes": rows + lists + 8 * n, "flops": fwd}
    n, sequences = case["n"] - case["tail"], case["sequences"]
    token = 4 + 4 * case["ref"] + (case["prompt"] > 0.0)
    if op.startswith("policy"):
        token += 4 + 4 * case["per_token"]
        sides = 4 * (sequences + 1) + 16 * sequences + 4 * sequences * (not case["per_token"])
    else:
        sides = 4 * (sequences + 1) + 12 * sequences
    if step:
        return {"bytes": (token + 4) * n + sides + 4 * sequences, "flops": 40 * n}
    return {"bytes": token * n + sides, "flops": 20 * n}


# ------------------------------------------------------------------- exact

def _exact_distill(case, s):
    n, dim, top = case["n"], case["dim"], case["top"]
    step = case["op"] == "distill_step"
    w = s["weight"].double()
    loss = torch.zeros(n, dtype=torch.float64, device="cuda")
    lse = torch.empty_like(loss)
    logp = torch.zeros(n, top, dtype=torch.float64, device="cuda")
    if step:
        dh = torch.empty(n, dim, dtype=torch.float64, device="cuda")
        dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    for r0 in range(0, n, 1024):
        r1 = min(n, r0 + 1024)
        h = s["hidden"][r0:r1].double()
        logits = torch.mm(h, w.t()) / case["temperature"]
        lse[r0:r1] = torch.logsumexp(logits, 1)
        row, col = (s["ids"][r0:r1] >= 0).nonzero(as_tuple=True)
        at = s["ids"][r0:r1][row, col]
        lp = logits[row, at] - lse[r0:r1][row]
        logp[r0 + row, col] = lp
        z = torch.full((r1 - r0, top), -math.inf, dtype=torch.float64, device="cuda")
        z[row, col] = s["teacher"][r0:r1].double()[row, col] / case["temperature"]
        logq = torch.log_softmax(z, 1)[row, col]
        loss.index_put_((r0 + row,), logq.exp() * (logq - lp), accumulate=True)
        if step:
            g = torch.softmax(logits, 1)
            g.index_put_((row, at), -logq.exp(), accumulate=True)
            scale = torch.zeros(r1 - r0, dtype=torch.float64, device="cuda")
            scale[row] = s["dloss"][r0:r1].double()[row] / case["temperature"]
            g.mul_(scale.unsqueeze(1))
            dh[r0:r1] = torch.mm(g, w)
            dw.addmm_(g.t(), h)
    return (loss, lse, logp, dh, dw) if step else (loss, lse, logp)


def _host(t, dtype=np.float64):
    return t.cpu().numpy().astype(dtype)


def _by_sequence(values, off):
    """Sums over [off[s], off[s + 1]), 0 for an empty one."""
    out = np.zeros(off.size - 1)
    full = np.flatnonzero(off[1:] > off[:-1])
    if full.size:
        out[full] = np.add.reduceat(values[:off[-1]], off[full])
    return out


def _exact_sequences(case, s):
    off = _host(s["offsets"], np.int64)
    inside = off[-1]
    length = np.diff(off)
    seq = np.repeat(np.arange(length.size), length)
    use = np.ones(inside, bool) if s["mask"] is None else _host(s["mask"], bool)[:inside]
    nll = _host(s["nll"])[:inside]
    ref = _host(s["ref"])[:inside] if case["ref"] else None
    count = _by_sequence(use.astype(np.float64), off)
    part = 1.0 / np.maximum(count, 1.0) if case["mean"] else np.ones_like(count)
    grad = np.zeros(case["n"])
    if case["op"].startswith("policy"):
        a = _host(s["advantages"])
        a = a[:inside] if case["per_token"] else a[seq]
        r = np.exp(_host(s["old"])[:inside] - nll)
        bound = np.where(a > 0, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW)
        cut = use & (((a > 0) & (r > bound)) | ((a < 0) & (r < bound)))
        token = -np.where(cut, bound, r) * a
        slope = np.where(cut, 0.0, r * a)
        kl = np.zeros_like(nll)
        if ref is not None:
            kl = np.expm1(nll - ref) - (nll - ref)
            token += KL_WEIGHT * kl
            slope += KL_WEIGHT * np.expm1(nll - ref)
        outs = [_by_sequence(np.where(use, token, 0.0), off) * part,
                _by_sequence(np.where(use, kl, 0.0), off) * part, count.astype(np.int32),
                _by_sequence(cut.astype(np.float64), off).astype(np.int32)]
        grad[:inside] = np.where(use, slope * (_host(s["dloss"]) * part)[seq], 0.0)
    else:
        beta, e = BETA[case["mean"]], case["smoothing"]
        reward = beta * part * _by_sequence(np.where(use, (0.0 if ref is None else ref) - nll, 0.0),
                                            off)
        x = reward[0::2] - reward[1::2] - MARGIN[case["mean"]]
        if case["kind"] == "logistic":
            loss = (1.0 - e) * np.logaddexp(0.0, -x) + e * np.logaddexp(0.0, x)
            slope = e / (1.0 + np.exp(-x)) - (1.0 - e) / (1.0 + np.exp(x))
        elif case["kind"] == "hinge":
            loss, slope = np.maximum(0.0, 1.0 - x), np.where(x < 1.0, -1.0, 0.0)
        else:
            loss, slope = np.square(1.0 - x), -2.0 * (1.0 - x)
        pair = (count[0::2] > 0) & (count[1::2] > 0)
        outs = [np.where(pair, loss, 0.0), x, reward, count.astype(np.int32)]
        by = np.where(pair, slope * _host(s["dloss"]), 0.0)
        each = np.empty(length.size)
        each[0::2], each[1::2] = -beta * by, beta * by
        grad[:inside] = np.where(use, (each * part)[seq], 0.0)
    if case["op"].endswith("step"):
        outs.append(grad)
    return tuple(torch.from_numpy(np.ascontiguousarray(o)) for o in outs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("distill"):
        return _exact_distill(case, s)
    return _exact_sequences(case, s)
