"""More operators that are measured: the cases, their inputs, and each operator's plain form
beside the framework's calls.

A vocabulary table [V, D] at both ends of a model:

* ``embed``   rows of the table times a scale, and the table's gradient:
                  out_n = s W[i_n]        dW_v = s sum over n with i_n = v of dout_n
              (the row ``padding`` gets no gradient).  The table is float, or int8 rows with a
              scale t_v each: W_v = q_v t_v.
* ``prefer``  a preference loss over pairs of sequences, through the table as output head.
              With z_iv = <hidden_i, W_v>, l_i = z_i,t(i) - log sum_v exp z_iv and h_j the sum
              (or the mean) over sequence j's positions of l_i - reference_i,
              x_p = h_p - h_{P + p} (sequences 0 .. P - 1 are preferred to P .. 2 P - 1):
                  sigmoid  -(1 - e) log S(b x - m) - e log S(m - b x),  S(y) = 1 / (1 + exp -y)
                  hinge    max(0, 1 - (b x - m))
                  square   (x - 1 / (2 b))^2
* ``policy``  the clipped policy loss with a KL term, through the same head.  With
              l_i = log softmax(z_i / T) at the action, r = exp(l_i - old_i),
              d = reference_i - l_i and A the advantage:
                  loss_i = -min(r A, clip(r, 1 - lo, 1 + hi) A) + c (exp d - d - 1)
              Both: dL/dz_iv = dL/dl_i ([v = t(i)] - p_iv) / T, dL/dhidden = dL/dz W,
              dL/dW = dL/dz^T hidden.  Positions whose target is IGNORE or that lie behind the
              last sequence do not count.
* ``int8``    the head's logits in 8-bit integers, a scale for each token and each row:
                  s_i = max |hidden_i| / 127, q_i = round(hidden_i / s_i) (to even),
                  out_iv = s_i t_v sum_k q_ik w_vk
"""
import math
import random

import torch

own = False

_DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
IGNORE = -100


def _embed(name, direction, n, v, d, dtype, table, scale=1.0, padded=0.0):
    return {"name": name, "op": "embed", "direction": direction, "n": n, "v": v, "d": d,
            "dtype": dtype, "table": table, "scale": scale, "padded": padded}


def _prefer(name, direction, pairs, n, v, d, dtype, reduction="mean", prompt=0.0, kind="sigmoid",
            beta=0.1, smoothing=0.0, margin=0.0, average=False, tail=0, reference=True):
    return {"name": name, "op": "prefer", "direction": direction, "pairs": pairs, "n": n, "v": v,
            "d": d, "dtype": dtype, "reduction": reduction, "prompt": prompt, "kind": kind,
            "beta": beta, "smoothing": smoothing, "margin": margin, "average": average,
            "tail": tail, "reference": reference}


def _policy(name, direction, n, v, d, dtype, reduction="mean", prompt=0.0, kl=0.0, low=0.2,
            high=0.2, temperature=1.0):
    return {"name": name, "op": "policy", "direction": direction, "n": n, "v": v, "d": d,
            "dtype": dtype, "reduction": reduction, "prompt": prompt, "kl": kl, "low": low,
            "high": high, "temperature": temperature}


def _int8(name, n, v, d, dtype):
    return {"name": name, "op": "int8", "direction": "forward", "n": n, "v": v, "d": d,
            "dtype": dtype}


def listed():
    return [
        # the next tokens of 8 requests looked up in a table served in int8: the smallest call
        _embed("embed_serve_8", "forward", 8, 32000, 2048, "bf16", "int8", 2048 ** 0.5),
        # a short fp32 training batch, odd sizes throughout
        _embed("embed_train_odd", "train", 333, 10007, 515, "fp32", "float", 515 ** 0.5, 0.2),
        # an ordinary training batch, a fourth of it padding
        _embed("embed_train_4096", "train", 4096, 32000, 2048, "bf16", "float", 1.0, 0.25),
        # a full training batch of a wide model with a large vocabulary
        _embed("embed_train_large", "train", 65536, 131072, 4096, "bf16", "float", 64.0, 0.05),
        # a few short pairs, odd sizes, per-pair losses
        _prefer("prefer_train_odd", "train", 3, 421, 10007, 515, "fp16", "none", 0.3,
                smoothing=0.1, tail=13),
        # validation: losses of 32 pairs, without a reference, length-normalised with a margin
        _prefer("prefer_eval", "forward", 32, 2000, 50000, 1536, "bf16", "mean", 0.5, beta=2.0,
                margin=0.5, average=True, reference=False),
        # an ordinary step over a large vocabulary; prompts do not count
        _prefer("prefer_train_large", "train", 16, 4096, 131072, 2048, "bf16", "mean", 0.4),
        # the loss of a few tokens while sampling, fp32
        _policy("policy_eval_fp32", "forward", 64, 32000, 1024, "fp32", "none", 0.0, 0.1),
        # an ordinary step, half of the positions being prompts
        _policy("policy_train_4096", "train", 4096, 32000, 2048, "bf16", "mean", 0.5, 0.04, 0.2,
                0.28),
        # a large step at a sampling temperature
        _policy("policy_train_large", "train", 8000, 131072, 4096, "bf16", "mean", 0.1, 0.0, 0.2,
                0.2, 0.8),
        # one token's logits while serving
        _int8("int8_logits_1", 1, 32000, 1024, "bf16"),
        # prompts scored in one call
        _int8("int8_logits_4096", 4096, 50021, 2048, "fp16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "prefer", "policy", "int8"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    train = rng.choice(["forward", "train", "train"])
    while True:
        n = _log_uniform(rng, 1, 65536 if op == "embed" else 8192)
        v = _log_uniform(rng, 1000, 131072)
        d = _log_uniform(rng, 16 if op == "embed" else 64, 4096)
        if rng.random() < 0.6:  # most widths and vocabularies are round, some are not
            d = max(64, d // 64 * 64)
            v = max(1000, v // 8 * 8)
        size = 4 if dtype == "fp32" else 2
        if op == "embed":
            if (2 * n + v) * d * size <= 2 ** 31:
                break
        # half the largest listed case in 16 bits; fp32 products are held to a fourth of that
        elif n * v * d <= (2 ** 41 if size == 2 else 2 ** 39) and \
                (op != "int8" or n * v * size <= 2 ** 29):
            break
    if op == "embed":
        table = "float" if train == "train" else rng.choice(["float", "int8"])
        c = _embed("", train, n, v, d, dtype, table, rng.choice([1.0, d ** 0.5]),
                   rng.choice([0.0, 0.05, 0.3]))
    elif op == "prefer":
        pairs = _log_uniform(rng, 1, max(1, min(64, n // 2)))
        n = max(n, 2 * pairs)
        kind = rng.choice(["sigmoid", "sigmoid", "hinge", "square"])
        c = _prefer("", train, pairs, n, v, d, dtype, rng.choice(["none", "sum", "mean"]),
                    rng.choice([0.0, 0.4]), kind, rng.choice([0.1, 0.5]),
                    rng.choice([0.0, 0.1]) if kind == "sigmoid" else 0.0,
                    rng.choice([0.0, 0.3]) if kind != "square" else 0.0,
                    rng.random() < 0.3, rng.choice([0, n // 50]), rng.random() < 0.8)
    elif op == "policy":
        c = _policy("", train, n, v, d, dtype, rng.choice(["none", "sum", "mean"]),
                    rng.choice([0.0, 0.1, 0.5]), rng.choice([0.0, 0.04]), 0.2,
                    rng.choice([0.2, 0.28]), rng.choice([1.0, 0.7]))
    else:
        c = _int8("", n, v, d, dtype)
    del c["name"]
    return c


def _lengths(case):
    """The 2 P sequences' lengths, ragged, and together all positions but the tail."""
    rng = random.Random("%(pairs)d %(n)d %(v)d %(d)d" % case)
    total, count = case["n"] - case["tail"], 2 * case["pairs"]
    if total < count:
        total = case["n"]
    weight = [rng.uniform(0.3, 1.0) for _ in range(count)]
    whole = sum(weight)
    sizes = [1 + int((total - count) * w / whole) for w in weight]
    sizes[rng.randrange(count)] += total - sum(sizes)
    return sizes


def _ignored(case):
    """Which positions do not count, as a list of truth values."""
    n, share = case["n"], case["prompt"]
    if case["op"] == "prefer":
        sizes = _lengths(case)
        return [k < min(size - 1, int(size * share)) for size in sizes for k in range(size)] \
            + [True] * (n - sum(sizes))
    run = min(97, n)  # sequences of that length, each with its prompt
    return [n > 1 and i % run < int(run * share) for i in range(n)]


def _int8_rows(x):
    """Rows in 8 bits with a scale each, rows a multiple of 16 bytes apart."""
    v, d = x.shape
    scales = x.abs().amax(1) / 127.0
    values = torch.zeros(v, (d + 15) // 16 * 16, dtype=torch.int8, device=x.device)
    values[:, :d] = torch.round(x / scales[:, None]).to(torch.int8)
    return values[:, :d], scales


def _log_probabilities(hidden, weight, target, temperature):
    """Of the targets, in the inputs' type: what an earlier version of the model gave them."""
    def part(h, t):
        z = (h @ weight.t()).float() / temperature
        return z.gather(1, t[:, None])[:, 0] - torch.logsumexp(z, 1)
    return torch.cat([part(h, t) for h, t in zip(hidden.split(1024), target.split(1024))])


def prepare(case, seed):
    n, v, d = case["n"], case["v"], case["d"]
    dt = _DTYPE[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    train = case["direction"] == "train"
    # rows of unit norm on average; low rows are the frequent ones
    weight = torch.empty(v, d, device="cuda").normal_(0, 1.0, generator=g).mul_(d ** -0.5)
    target = (v * torch.rand(n, device="cuda", generator=g) ** 3).long().clamp_(max=v - 1)
    state = {"case": case}
    if case["op"] == "embed":
        if case["table"] == "int8":
            state["values"], state["scales"] = _int8_rows(weight)
        else:
            state["weight"] = weight.to(dt)
        state["padding"] = v - 1
        target[torch.rand(n, device="cuda", generator=g) < case["padded"]] = v - 1
        state["indices"] = target
        if train:
            state["upstream"] = torch.randn(n, d, device="cuda", generator=g).to(dt)
        return state
    # hidden states of which some already point to their target
    hidden = torch.randn(n, d, device="cuda", generator=g)
    hidden += weight[target] * (14.0 * torch.rand(n, 1, device="cuda", generator=g))
    hidden = hidden.to(dt)
    if case["op"] == "int8":
        state["hidden"] = hidden
        state["values"], state["scales"] = _int8_rows(weight)
        return state
    weight = weight.to(dt)
    state["hidden"] = hidden.requires_grad_(train)
    state["weight"] = weight.requires_grad_(train)
    temperature = case.get("temperature", 1.0)
    with torch.no_grad():
        logp = _log_probabilities(hidden, weight, target, temperature)
    noise = torch.randn(2, n, device="cuda", generator=g)
    target[torch.tensor(_ignored(case), device="cuda")] = IGNORE
    state["targets"] = target
    if case["op"] == "prefer":
        sizes = torch.tensor(_lengths(case), device="cuda")
        zero = torch.zeros(1, dtype=torch.int64, device="cuda")
        state["offsets"] = torch.cat([zero, sizes.cumsum(0)])
        # the model has moved from the reference, some sequences more than others
        drift = 0.2 * torch.randn(sizes.numel(), device="cuda", generator=g)
        drift = torch.cat([drift.repeat_interleave(sizes), drift.new_zeros(n)])[:n]
        state["reference"] = logp + drift + 0.3 * noise[0] if case["reference"] else None
        count = case["pairs"]
    else:
        # one advantage per sequence, old probabilities around the clip bounds
        adv = torch.randn((n + 96) // 97, device="cuda", generator=g)
        state["advantages"] = adv.repeat_interleave(97)[:n].contiguous()
        state["old"] = logp + 0.2 * noise[0]
        state["reference"] = logp + 0.3 * noise[1] if case["kl"] else None
        count = n
    if case["reduction"] == "none" and train:
        state["upstream"] = 0.1 + torch.rand(count, device="cuda", generator=g)
    return state


def _run_own(state):
    case = state["case"]
    if case["op"] == "embed":
        from tensor_train_compressed_ttembeddingbag_amd import embedding as E
        if case["table"] == "int8":
            from tensor_train_compressed_ttembeddingbag_amd.quant import Int8Rows
            table = Int8Rows(state["values"], state["scales"])
            return E.embedding(state["indices"], table, scale=case["scale"],
                               dtype=_DTYPE[case["dtype"]])
        out = E.embedding(state["indices"], state["weight"], scale=case["scale"],
                          padding_idx=state["padding"])
        if case["direction"] == "forward":
            return out
        return out, E.embedding_gradient(state["upstream"], state["indices"], case["v"],
                                         scale=case["scale"], padding_idx=state["padding"])
    if case["op"] == "int8":
        from tensor_train_compressed_ttembeddingbag_amd.quant import Int8Rows, int8_linear
        return int8_linear(state["hidden"], Int8Rows(state["values"], state["scales"]))
    from tensor_train_compressed_ttembeddingbag_amd import loss as L
    if case["op"] == "prefer":
        out, more = L.linear_preference(
            state["hidden"], state["weight"], state["targets"], state["offsets"],
            state["reference"], beta=case["beta"], kind=case["kind"],
            label_smoothing=case["smoothing"], margin=case["margin"], average=case["average"],
            ignore_index=IGNORE, reduction=case["reduction"], return_ratios=True)
    else:
        out, more = L.linear_policy(
            state["hidden"], state["weight"], state["targets"], state["advantages"],
            state["old"], state["reference"], clip_low=case["low"], clip_high=case["high"],
            kl_coef=case["kl"], temperature=case["temperature"], ignore_index=IGNORE,
            reduction=case["reduction"], return_logps=True)
    if case["direction"] == "forward":
        return out, more
    dh, dw = torch.autograd.grad(out, (state["hidden"], state["weight"]), state.get("upstream"))
    return out.detach(), more, dh, dw


def _plain_embed(state):
    case, i = state["case"], state["indices"]
    if case["table"] == "int8":
        rows = state["values"][i].float() * state["scales"][i][:, None]
        return (rows * case["scale"]).to(_DTYPE[case["dtype"]])
    weight = state["weight"]
    out = (weight[i].float() * case["scale"]).to(weight.dtype)
    if case["direction"] == "forward":
        return out
    up = state["upstream"].float() * (case["scale"] * (i != state["padding"]).float())[:, None]
    dw = torch.zeros(weight.shape, device=weight.device).index_add_(0, i, up)
    return out, dw.to(weight.dtype)


def _plain_int8(state):
    x, w = state["hidden"].float(), state["values"].float()
    s = x.abs().amax(1, keepdim=True) / 127.0
    q = torch.round(x / torch.where(s > 0, s, 1.0))
    return ((q @ w.t()) * s * state["scales"]).to(state["hidden"].dtype)


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    with torch.no_grad():
        if case["op"] == "embed":
            return _plain_embed(state)
        if case["op"] == "int8":
            return _plain_int8(state)
        t, n = state["targets"], case["n"]
        h, w = state["hidden"].float(), state["weight"].float()
        temp = case.get("temperature", 1.0)
        z = h @ w.t()
        if temp != 1.0:
            z /= temp
        valid = t != IGNORE
        pick = torch.where(valid, t, 0)[:, None]
        m = z.amax(1, keepdim=True)
        lse = m[:, 0] + torch.exp(z - m).sum(1).log()
        logp = torch.where(valid, z.gather(1, pick)[:, 0] - lse, 0.0)
        far = logp.double()  # sums of many terms, and ratios next to a bound
        if case["op"] == "prefer":
            off, pairs, b = state["offsets"], case["pairs"], case["beta"]
            seq = torch.bucketize(torch.arange(n, device=t.device), off, right=True) - 1
            inside = seq < 2 * pairs
            seq = torch.where(inside, seq, 0)
            valid = valid & inside
            per = far - state["reference"] if case["reference"] else far
            per = torch.where(valid, per, 0.0)
            ratio = per.new_zeros(2 * pairs).index_add_(0, seq, per)
            share = torch.ones_like(ratio)
            if case["average"]:
                kept = torch.zeros_like(ratio).index_add_(0, seq, valid.double())
                share = 1.0 / kept.clamp(min=1)
            ratio = ratio * share
            x = ratio[:pairs] - ratio[pairs:]
            if case["kind"] == "square":
                gap = x - 1.0 / (2.0 * b)
                rows, slope = gap * gap, 2.0 * gap
            else:
                y = b * x - case["margin"]
                if case["kind"] == "hinge":
                    rows, slope = torch.relu(1.0 - y), -b * (y < 1.0).double()
                else:
                    e = case["smoothing"]
                    low = torch.log1p(torch.exp(-y.abs()))  # -log S(y) = low + max(0, -y)
                    rows = low + (1 - e) * torch.relu(-y) + e * torch.relu(y)
                    slope = b * (torch.sigmoid(y) - (1 - e))
            count = pairs
            more = ratio.float().view(2, pairs)
        else:
            adv = state["advantages"].double()
            r = torch.exp(far - state["old"])
            free, held = r * adv, r.clamp(1 - case["low"], 1 + case["high"]) * adv
            rows = -torch.minimum(free, held)
            slope = -torch.where(free <= held, free, 0.0)
            if case["kl"]:
                dist = state["reference"] - far
                rows = rows + case["kl"] * (torch.expm1(dist) - dist)
                slope = slope - case["kl"] * torch.expm1(dist)
            rows = torch.where(valid, rows, 0.0)
            count = valid.sum().clamp(min=1)
            more = logp
        if case["reduction"] == "none":
            out = rows.float()
        else:
            out = (rows.sum() / (count if case["reduction"] == "mean" else 1)).float()
        if case["direction"] == "forward":
            return out, more
        c = slope
        if case["reduction"] == "none":
            c = c * state["upstream"]
        elif case["reduction"] == "mean":
            c = c / count
        if case["op"] == "prefer":
            c = torch.cat([c, -c]) * share
            c = c[seq]
        c = torch.where(valid, c, 0.0).float() / temp
        z -= lse[:, None]
        z.exp_()
        z.scatter_add_(1, pick, torch.full_like(c, -1.0)[:, None])
        z *= -c[:, None]
        dt = state["hidden"].dtype
        return out, more, (z @ w).to(dt), (z.t() @ h).to(dt)


def exact(case, seed):
    """The definitions in 64 bits, a block of positions at a time."""
    state = prepare(case, seed)
    n, v, d = case["n"], case["v"], case["d"]
    train = case["direction"] == "train"
    with torch.no_grad():
        if case["op"] == "embed":
            i = state["indices"]
            if case["table"] == "int8":
                table = state["values"].double() * state["scales"].double()[:, None]
                return table.index_select(0, i) * case["scale"]
            out = state["weight"].index_select(0, i).double() * case["scale"]
            if not train:
                return out
            live = torch.nonzero(i != state["padding"])[:, 0]
            dw = torch.zeros(v, d, dtype=torch.float64, device="cuda")
            dw.index_add_(0, i[live], state["upstream"][live].double(), alpha=case["scale"])
            return out, dw
        if case["op"] == "int8":
            out = torch.empty(n, v, dtype=torch.float64, device="cuda")
            wt = state["values"].double().t().contiguous()
            for a in range(0, n, 1024):
                x = state["hidden"][a:a + 1024].double()
                s = x.abs().max(1, keepdim=True).values / 127
                q = (x / s.clamp(min=1e-300)).round()
                out[a:a + 1024] = torch.mm(q, wt) * (s * state["scales"].double()[None])
            return out
        w = state["weight"].detach().double()
        wt = w.t().contiguous()
        temp = case.get("temperature", 1.0)
        flags = torch.tensor(_ignored(case), device="cuda")
        kept = torch.nonzero(~flags)[:, 0]
        block = max(1, 2 ** 27 // v)
        logp = torch.zeros(n, dtype=torch.float64, device="cuda")
        for a in range(0, kept.numel(), block):
            pos = kept[a:a + block]
            x = torch.log_softmax(torch.mm(state["hidden"][pos].double(), wt) / temp, 1)
            logp[pos] = x[torch.arange(pos.numel(), device="cuda"), state["targets"][pos]]
        leaf = logp.clone().requires_grad_(train)
        with torch.enable_grad():
            if case["op"] == "prefer":
                per = leaf - state["reference"].double() if case["reference"] else leaf
                ends = [int(e) for e in state["offsets"].tolist()]
                sums = []
                for a, e in zip(ends, ends[1:]):
                    part = per[a:e][~flags[a:e]]
                    sums.append(part.mean() if case["average"] else part.sum())
                ratio = torch.stack(sums)
                x = ratio[:case["pairs"]] - ratio[case["pairs"]:]
                y = case["beta"] * x - case["margin"]
                if case["kind"] == "square":
                    rows = (x - 0.5 / case["beta"]) ** 2
                elif case["kind"] == "hinge":
                    rows = torch.clamp(1 - y, min=0)
                else:
                    e = case["smoothing"]
                    rows = (1 - e) * torch.nn.functional.softplus(-y) \
                        + e * torch.nn.functional.softplus(y)
                more, count = ratio.detach().view(2, -1), case["pairs"]
            else:
                r = torch.exp(leaf - state["old"].double())
                adv = state["advantages"].double()
                rows = -torch.min(r * adv, torch.clamp(r, 1 - case["low"], 1 + case["high"]) * adv)
                if case["kl"]:
                    dist = state["reference"].double() - leaf
                    rows = rows + case["kl"] * (torch.exp(dist) - 1 - dist)
                rows = rows.masked_fill(flags, 0.0)
                more, count = logp, max(1, kept.numel())
            out = rows if case["reduction"] == "none" else rows.sum()
            if case["reduction"] == "mean":
                out = out / count
            if not train:
                return out, more
            up = state["upstream"].double() if case["reduction"] == "none" else None
            coef = torch.autograd.grad(out, leaf, up)[0] / temp
        dh = torch.zeros(n, d, dtype=torch.float64, device="cuda")
        dw = torch.zeros(v, d, dtype=torch.float64, device="cuda")
        for a in range(0, kept.numel(), block):
            pos = kept[a:a + block]
            h = state["hidden"][pos].double()
            dz = -torch.softmax(torch.mm(h, wt) / temp, 1)
            dz[torch.arange(pos.numel(), device="cuda"), state["targets"][pos]] += 1
            dz *= coef[pos, None]
            dh[pos] = torch.mm(dz, w)
            dw += torch.mm(dz.t().contiguous(), h)
        return out.detach(), more, dh, dw


def work(case):
    """Each input read once and each output written once (of a table that is looked up, the
    rows asked for); products over the positions that count, once forward and (training) once
    for each of the two gradients."""
    n, v, d = case["n"], case["v"], case["d"]
    size = 4 if case["dtype"] == "fp32" else 2
    train = case["direction"] == "train"
    if case["op"] == "embed":
        row = d + 4 if case["table"] == "int8" else d * size
        data = 8 * n + min(n, v) * row + n * d * size
        if train:
            data += (n + v) * d * size
        return {"bytes": data, "flops": (2 if train else 1) * n * d}
    if case["op"] == "int8":
        return {"bytes": n * d * size + v * (d + 4) + n * v * size, "flops": 2 * n * v * d}
    kept = n - sum(_ignored(case))
    data = (kept * d + v * d) * size + n * 8
    if case["op"] == "prefer":
        rows, more = case["pairs"], 2 * case["pairs"]
        data += 4 * n * bool(case["reference"])
    else:
        rows = more = n
        data += 4 * n * (3 if case["kl"] else 2)
    data += 4 * (rows if case["reduction"] == "none" else 1) + 4 * more
    if train:
        data += (n * d + v * d) * size + (4 * rows if case["reduction"] == "none" else 0)
    return {"bytes": data, "flops": (6 if train else 2) * kept * v * d}
