"""What a language model adds at the two ends of a gradient-bucket step, as measurable calls.

Three operators, each in a plain form (elementary torch operations in 32 bits, rounded once at the
end) and as calls of this package (``own = True``):

* ``clip``        the global norm over many gradient tensors and the clipped gradients;
* ``embed``       the embedding lookup with its scale, and ``embed_grad``, the table's gradient;
* ``loss_eval``   softmax cross entropy of hidden states against a vocabulary projection (losses and
                  log-sum-exps), and ``loss_step``, the same with the gradients of both inputs.

A case is a dict of plain values; ``prepare`` makes a case's inputs on the GPU from a seed.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
IGNORE = -100


def tensor_sizes(layers, width, vocab):
    """The gradient tensors of a transformer: the embedding table, then sixteen tensors a layer."""
    layer = [width * width, width] * 4 + [width, width] + [4 * width * width, 4 * width, 4 * width * width, width] + \
        [width, width]
    return [vocab * width] + layers * layer


def listed():
    return [
        # a small model's seventeen tensors: latency decides
        {"name": "clip_small_f32", "op": "clip", "layers": 1, "width": 128, "vocab": 1000, "dtype": "f32",
         "norm": 2, "max_norm": 1.0},
        # the gradients of GPT-2 small as bf16 tensors, 193 of them, packed tight
        {"name": "clip_gpt2_bf16", "op": "clip", "layers": 12, "width": 768, "vocab": 50257, "dtype": "bf16",
         "norm": 2, "max_norm": 1.0},
        # BERT-large's reduced fp32 gradients: 1.3 GB, far beyond L2
        {"name": "clip_bert_f32", "op": "clip", "layers": 24, "width": 1024, "vocab": 30522, "dtype": "f32",
         "norm": 2, "max_norm": 1.0},
        # the token a decoder has just produced
        {"name": "embed_one_bf16", "op": "embed", "tokens": 1, "vocab": 50257, "dim": 768, "dtype": "bf16"},
        # a training batch of 8 sequences of 1024 tokens
        {"name": "embed_batch_f32", "op": "embed", "tokens": 8192, "vocab": 50257, "dim": 768, "dtype": "f32"},
        # that batch's embedding gradient: most of the table's rows are zero
        {"name": "embed_grad_gpt2_bf16", "op": "embed_grad", "tokens": 8192, "vocab": 50257, "dim": 768,
         "dtype": "bf16", "padded": 0.0},
        # a long batch padded to a fixed length, ragged token count, fp16, a third of it padding
        {"name": "embed_grad_long_f16", "op": "embed_grad", "tokens": 65521, "vocab": 30522, "dim": 1024,
         "dtype": "f16", "padded": 0.3},
        # scoring one token against the whole vocabulary
        {"name": "loss_eval_one_bf16", "op": "loss_eval", "tokens": 1, "vocab": 50257, "dim": 768, "dtype": "bf16",
         "ignored": 0.0},
        # evaluating a document of ragged length, fp16
        {"name": "loss_eval_ragged_f16", "op": "loss_eval", "tokens": 1999, "vocab": 50257, "dim": 768,
         "dtype": "f16", "ignored": 0.0},
        # a GPT-2 small training batch: 8 x 1024 tokens against 50257 words
        {"name": "loss_step_gpt2_bf16", "op": "loss_step", "tokens": 8192, "vocab": 50257, "dim": 768,
         "dtype": "bf16", "ignored": 0.0},
        # masked-word training at BERT-large's sizes: 15% of the tokens carry a target
        {"name": "loss_step_masked_f16", "op": "loss_step", "tokens": 8192, "vocab": 30522, "dim": 1024,
         "dtype": "f16", "ignored": 0.85},
        # a wide model with a large vocabulary: three products of 4.4 TFLOP
        {"name": "loss_step_wide_bf16", "op": "loss_step", "tokens": 4096, "vocab": 131072, "dim": 4096,
         "dtype": "bf16", "ignored": 0.02},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["clip", "clip", "embed", "embed_grad", "embed_grad", "loss_eval", "loss_step", "loss_step"])
    if op == "clip":
        while True:
            c = {"op": op, "layers": _spread(rng, 1, 24), "width": _spread(rng, 64, 1280),
                 "vocab": _spread(rng, 1000, 60000), "dtype": rng.choice(["f32", "bf16", "f16"]),
                 "norm": rng.choice([2, 2, 0]), "max_norm": rng.choice([1e-3, 0.5, 1.0, 1e6])}
            if sum(tensor_sizes(c["layers"], c["width"], c["vocab"])) <= 330_000_000:
                return c
    c = {"op": op, "tokens": _spread(rng, 1, 65536 if op.startswith("embed") else 16384),
         "vocab": _spread(rng, 1000, 131072), "dim": 0, "dtype": ""}
    # dimensions in steps of 8 mostly, and odd ones
    c["dim"] = _spread(rng, 64, 4096)
    if rng.random() < 0.7:
        c["dim"] = c["dim"] // 8 * 8
    if c["dim"] == 3072:
        c["dim"] += 8
    if op == "embed":
        c["dtype"] = rng.choice(["f32", "bf16", "f16"])
    elif op == "embed_grad":
        c["dtype"] = rng.choice(["f32", "bf16", "f16"])
        c["padded"] = rng.choice([0.0, 0.0, 0.5])
    else:
        c["dtype"] = rng.choice(["bf16", "bf16", "f16"])
        c["ignored"] = rng.choice([0.0, 0.1, 0.85])
        while c["tokens"] * c["vocab"] * c["dim"] > 4096 * 131072 * 4096:
            c["tokens"] = c["tokens"] // 2 + 1
    return c


def _ids(count, vocab, gen):
    """Token ids whose frequencies fall like one over their rank, as words' do."""
    u = torch.rand(count, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    st = {"case": dict(case), "op": op, "dtype": dt}
    if op == "clip":
        sizes = tensor_sizes(case["layers"], case["width"], case["vocab"])
        # gradients packed tight, as in a bucket, each tensor with a magnitude of its own
        flat = torch.randn(sum(sizes), generator=gen, device="cuda", dtype=torch.float32)
        views = torch.split(flat, sizes)
        torch._foreach_mul_(list(views), [1e-3 * (1.0 + (k * 7 % 5)) for k in range(len(sizes))])
        flat = flat.to(dt)
        out = torch.empty_like(flat)
        st.update(flat=flat, out=out, max_norm=float(case["max_norm"]))
        if own:
            from allreduce_ddp_assign_gb300 import lm

            st["clipper"] = lm.GradClipper(list(torch.split(flat, sizes)), out=list(torch.split(out, sizes)),
                                           norm_type=2.0 if case["norm"] == 2 else math.inf)
        return st
    T, V, D = case["tokens"], case["vocab"], case["dim"]
    ids = _ids(T, V, gen)
    if op in ("embed", "embed_grad"):
        st["scale"] = math.sqrt(D)
        st["ids"] = ids
        if op == "embed":
            st["weight"] = torch.randn(V, D, generator=gen, device="cuda").mul_(0.02).to(dt)
            if own:
                from allreduce_ddp_assign_gb300 import lm

                st["table"] = lm.TokenEmbedding(V, D, dt, scale=st["scale"])
            return st
        st["padding"] = 0
        padded = int(case["padded"] * T)
        if padded:
            ids[T - padded:] = 0
        st["grad_out"] = torch.randn(T, D, generator=gen, device="cuda").mul_(1e-3).to(dt)
        if own:
            from allreduce_ddp_assign_gb300 import lm

            st["table"] = lm.TokenEmbedding(V, D, dt, scale=st["scale"], padding_idx=0)
        return st
    weight = torch.randn(V, D, generator=gen, device="cuda").mul_(0.02)
    hidden = torch.randn(T, D, generator=gen, device="cuda")
    # the model knows some of its targets: a part of the target's row in the hidden state
    knows = torch.rand(T, 1, generator=gen, device="cuda") * 12.0 / (0.0004 * D)
    hidden.addcmul_(weight[ids], knows)
    st["weight"], st["hidden"] = weight.to(dt), hidden.to(dt)
    dropped = torch.rand(T, generator=gen, device="cuda") < case["ignored"]
    st["targets"] = torch.where(dropped, torch.full_like(ids, IGNORE), ids)
    if op == "loss_step":
        # the gradient of the mean over the tokens that count, with a loss scale where the gradients are fp16
        valid = (~dropped).float()
        st["grad_loss"] = valid / valid.sum().clamp(min=1.0) * (1024.0 if dt == torch.float16 else 1.0)
    if own:
        from allreduce_ddp_assign_gb300 import lm

        st["loss"] = lm.VocabLoss(V, D, dt, ignore_index=IGNORE)
    return st


def _run_own(st):
    op = st["op"]
    if op == "clip":
        norm = st["clipper"].clip(st["max_norm"])
        return {"norm": norm, "clipped": st["out"]}
    if op == "embed":
        return {"out": st["table"].forward(st["weight"], st["ids"])}
    if op == "embed_grad":
        return {"grad_weight": st["table"].backward(st["grad_out"], st["ids"])}
    loss, lse = st["loss"].forward(st["hidden"], st["weight"], st["targets"])
    if op == "loss_eval":
        return {"loss": loss, "lse": lse}
    gh, gw = st["loss"].backward(st["hidden"], st["weight"], st["targets"], lse, st["grad_loss"])
    return {"loss": loss, "lse": lse, "grad_hidden": gh, "grad_weight": gw}


def run(st):
    if own:
        return _run_own(st)
    op, dt = st["op"], st["dtype"]
    if op == "clip":
        g = st["flat"].float()
        norm = g.square().sum().sqrt() if st["case"]["norm"] == 2 else g.abs().max()
        coef = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        st["out"].copy_(g * coef)
        return {"norm": norm.reshape(1), "clipped": st["out"]}
    if op == "embed":
        return {"out": (st["weight"][st["ids"]].float() * st["scale"]).to(dt)}
    if op == "embed_grad":
        c = st["case"]
        g = st["grad_out"].float() * st["scale"]
        g = g * (st["ids"] != st["padding"]).unsqueeze(1)
        gw = torch.zeros(c["vocab"], c["dim"], device="cuda").index_add_(0, st["ids"], g)
        return {"grad_weight": gw.to(dt)}
    h, w, t = st["hidden"].float(), st["weight"].float(), st["targets"]
    valid = t != IGNORE
    at = torch.where(valid, t, torch.zeros_like(t)).unsqueeze(1)
    z = h @ w.t()
    top = z.amax(dim=1, keepdim=True)
    lse = (z - top).exp_().sum(dim=1, keepdim=True).log() + top
    loss = lse - z.gather(1, at)
    zero = torch.zeros_like(loss[:, 0])
    res = {"loss": torch.where(valid, loss[:, 0], zero), "lse": torch.where(valid, lse[:, 0], zero)}
    if op == "loss_eval":
        return res
    z.sub_(lse).exp_()
    z.scatter_add_(1, at, torch.full_like(lse, -1.0))
    z.mul_(torch.where(valid, st["grad_loss"], zero).unsqueeze(1))
    res["grad_hidden"] = (z @ w).to(dt)
    res["grad_weight"] = (z.t() @ h).to(dt)
    return res


def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "clip":
        n = sum(tensor_sizes(case["layers"], case["width"], case["vocab"]))
        return {"bytes": 2 * n * b + 4, "flops": 3 * n}
    T, V, D = case["tokens"], case["vocab"], case["dim"]
    if op == "embed":
        return {"bytes": T * (2 * D * b + 8), "flops": T * D}
    if op == "embed_grad":
        return {"bytes": T * (D * b + 8) + V * D * b, "flops": 2 * T * D}
    # tokens without a target need no product
    n = max(1.0, T * (1.0 - case["ignored"]))
    bytes_, flops = (T * D + V * D) * b + 16 * T, 2.0 * n * V * D
    if op == "loss_step":
        bytes_, flops = bytes_ + (T * D + V * D) * b + 4 * T, 3 * flops
    return {"bytes": bytes_, "flops": flops}


def exact(case, seed):
    """The operators' definitions in 64 bits on the same inputs."""
    op = case["op"]
    if op in ("loss_eval", "loss_step"):
        products = 3 if op == "loss_step" else 1
        if 2.0 * case["tokens"] * case["vocab"] * case["dim"] * products > 9e12:
            return None
    st = prepare(case, seed)
    if op == "clip":
        g = st["flat"].double()
        norm = torch.linalg.vector_norm(g, ord=2 if case["norm"] == 2 else math.inf)
        return {"norm": norm.reshape(1), "clipped": g * min(1.0, st["max_norm"] / (float(norm) + 1e-6))}
    if op == "embed":
        return {"out": st["weight"].index_select(0, st["ids"]).double().mul_(st["scale"])}
    if op == "embed_grad":
        # sums over runs of equal ids: differences of a running sum of the sorted rows, a block of columns at a time
        V, D = case["vocab"], case["dim"]
        keep = (st["ids"] != st["padding"]).nonzero()[:, 0]
        ids, order = torch.sort(st["ids"][keep], stable=True)
        edges = torch.searchsorted(ids, torch.arange(V + 1, device="cuda"))
        gw = torch.empty(V, D, dtype=torch.float64, device="cuda")
        for c in range(0, D, 256):
            rows = st["grad_out"][keep[order], c:c + 256].double()
            total = torch.cat([torch.zeros_like(rows[:1]), rows.cumsum(0)]) if len(keep) else rows.new_zeros(1, min(256, D - c))
            gw[:, c:c + 256] = (total[edges[1:]] - total[edges[:-1]]) * st["scale"]
        return {"grad_weight": gw}
    T, V = case["tokens"], case["vocab"]
    w = st["weight"].double()
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    gh = torch.zeros(T, case["dim"], dtype=torch.float64, device="cuda")
    gw = torch.zeros_like(w)
    rows = (st["targets"] != IGNORE).nonzero()[:, 0]
    for part in torch.split(rows, 2048):
        h = st["hidden"][part].double()
        z = torch.mm(h, w.T)
        e = torch.logsumexp(z, dim=1)
        t = st["targets"][part]
        loss[part] = e - z[torch.arange(len(part), device="cuda"), t]
        lse[part] = e
        if op == "loss_step":
            g = torch.softmax(z, dim=1) - torch.nn.functional.one_hot(t, V)
            g = g * st["grad_loss"][part].double()[:, None]
            gh[part] = torch.mm(g, w)
            gw += torch.mm(g.T, h)
    if op == "loss_eval":
        return {"loss": loss, "lse": lse}
    return {"loss": loss, "lse": lse, "grad_hidden": gh, "grad_weight": gw}
