"""Code frames through a streaming transformer layer: quantizer, windowed attention with its gradient, paged cache.

    python examples/streaming_attention.py

Clips of latents are quantized (``rvq_encode``) and their codes embedded (``rvq_decode``), as a model over code frames
sees them. One attention layer with a bounded window and a few sinks then

1. trains: attention over all clips at once and one gradient step on its projection;
2. serves: the first frames of every clip go into a paged cache at once, the others frame by frame, as they would be
   generated. Half way every clip is forked into a second listener, the pages behind the window are given back, the
   first listeners leave and the pool is compacted.

What the cache gives frame by frame is compared with the attention over whole clips.
"""

import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import residual_vector_quantization_amd as rvq  # noqa: E402
import rvq_workloads as W  # noqa: E402

Q_HEADS, KV_HEADS, DIM = 8, 2, 64
WINDOW, SINKS, PAGE = 24, 2, 8


def offsets(lens, device):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=device)


def embed(lens, device):
    """Latents of the clips -> codes -> what the codes stand for, float32 [frames, 64]."""
    w = W.WORKLOADS["clip"]
    books = torch.from_numpy(W.codebooks(w.n_stages, w.n_codes, w.dim, w.decay, w.seed)).to(device)
    gen = torch.Generator().manual_seed(w.seed)
    x = torch.randn(sum(lens), w.dim, generator=gen).to(device)
    prepared = rvq.rvq_prepare_codebooks(books)
    codes, _, _ = rvq.rvq_encode_prepared(x, books, prepared, residual=False)
    return rvq.rvq_decode(codes, books)


def split_heads(qkv):
    return qkv[:, :Q_HEADS], qkv[:, Q_HEADS:Q_HEADS + KV_HEADS], qkv[:, Q_HEADS + KV_HEADS:]


def train_step(frames, weight, cu, target, rate):
    """One step on the projection: loss = mean square of (attention - target). Returns the loss and the new weight."""
    qkv = (frames.to(weight.dtype) @ weight).view(-1, Q_HEADS + 2 * KV_HEADS, DIM)
    q, k, v = split_heads(qkv)
    out, lse = rvq.rvq_window_attention(q, k, v, cu, window=WINDOW, sinks=SINKS)
    error = out.float() - target
    dout = (error * (2 / error.numel()) * 2.0 ** 12).to(out.dtype)          # loss scaling for float16
    dqkv = torch.empty_like(qkv)
    rvq.rvq_window_attention_backward(dout, q, k, v, out, lse, cu, window=WINDOW, sinks=SINKS, grads=split_heads(dqkv))
    dweight = frames.t() @ dqkv.view(dqkv.shape[0], -1).float() * 2.0 ** -12
    return error.square().mean(), (weight.float() - rate * dweight).to(weight.dtype)


def serve(qkv, lens, known, device):
    """Attention of every frame from ``known`` on, through the cache: [clips][frames][heads, dim]."""
    clips, cu = len(lens), torch.tensor(lens).cumsum(0).tolist()
    first = [c - n for c, n in zip(cu, lens)]
    cols = -(-max(lens) // PAGE)
    pages = 2 * clips * cols
    pools = [torch.zeros(1, pages, KV_HEADS, PAGE, DIM, dtype=qkv.dtype, device=device) for _ in range(2)]
    layer = [p[0] for p in pools]
    # two rows a clip: the listener from the start, and one that joins later
    table = torch.full((2 * clips, cols), -1, dtype=torch.int32, device=device)
    counts = torch.zeros(2 * clips, dtype=torch.int32, device=device)
    refs = torch.zeros(pages, dtype=torch.int32, device=device)
    q, k, v = split_heads(qkv)

    def admit(rows, new):
        """New frames (rows of k and v, and how many a listener) get their pages and are written."""
        nonlocal table, refs, counts
        more = torch.tensor(new, dtype=torch.int32, device=device)
        table, refs, missing = rvq.rvq_cache_reserve(table, counts, counts + more, refs, PAGE)
        rvq.rvq_cache_append(k[rows], v[rows], *layer, table, counts, offsets(new, device))
        counts = counts + more
        return missing

    missing = admit([first[b] + i for b in range(clips) for i in range(min(known, lens[b]))],
                    [min(known, n) for n in lens] + [0] * clips)
    got = [[] for _ in lens]
    at = clips                                # the listeners that hear: the first `clips` rows, later the others
    for i in range(known, max(lens)):
        active = [b for b in range(clips) if i < lens[b]]
        if i == (known + max(lens)) // 2:
            parents = torch.arange(clips, dtype=torch.int32, device=device)
            table, counts, refs, _ = rvq.rvq_cache_fork(table, counts, refs, parents, parents + clips, *pools)
            drop = torch.tensor([1] * clips + [0] * clips, dtype=torch.int32, device=device)
            table, counts, refs = rvq.rvq_cache_free(table, counts, refs, PAGE, drop=drop, window=WINDOW, sinks=SINKS)
            table, refs, live = rvq.rvq_cache_compact(table, refs, *pools)
            at = 2 * clips
        row_of = {b: b + at - clips for b in active}
        new = [0] * (2 * clips)
        for b in active:
            new[row_of[b]] = 1
        missing = missing + admit([first[b] + i for b in active], new)
        queries = torch.zeros(2 * clips, Q_HEADS, DIM, dtype=qkv.dtype, device=device)
        queries[[row_of[b] for b in active]] = q[[first[b] + i for b in active]]
        out = rvq.rvq_cache_attention(queries, *layer, table, counts, window=WINDOW, sinks=SINKS)
        for b in active:
            got[b].append(out[row_of[b]])
    return got, missing, live


def main(lens=(70, 33, 52), known=10, dtype=torch.bfloat16, steps=20, quiet=False):
    """Returns (losses, largest difference between cache and whole attention over the largest value, live pages)."""
    device = torch.device("cuda:0")
    lens = list(lens)
    frames, cu = embed(lens, device), offsets(lens, device)
    gen = torch.Generator().manual_seed(1)
    weight = (torch.randn(64, (Q_HEADS + 2 * KV_HEADS) * DIM, generator=gen) / math.sqrt(64)).to(device, dtype)
    target = torch.zeros(len(frames), Q_HEADS, DIM, device=device)
    losses = []
    for _ in range(steps):
        loss, weight = train_step(frames, weight, cu, target, rate=10.0)
        losses.append(loss.item())
    qkv = (frames.to(dtype) @ weight).view(-1, Q_HEADS + 2 * KV_HEADS, DIM)
    q, k, v = split_heads(qkv)
    whole, _ = rvq.rvq_window_attention(q, k, v, cu, window=WINDOW, sinks=SINKS)
    got, missing, live = serve(qkv, lens, known, device)
    worst, start = 0.0, 0
    for b, n in enumerate(lens):
        if got[b]:
            worst = max(worst, (torch.stack(got[b]).float() - whole[start + known:start + n].float()).abs().max().item())
        start += n
    worst /= v.abs().max().item()
    if not quiet:
        print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f} in {steps} steps; cache against whole clips: "
              f"{worst:.2e} of the largest value; pages missing {missing.item()}, in use after compaction {live.item()}")
    return losses, worst, missing.item(), live.item()


if __name__ == "__main__":
    main()
