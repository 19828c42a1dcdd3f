"""Decoding with a paged key-value cache: prompts of several lengths go in,
then tokens are generated a step at a time -- turn the queries, write the new
keys and values (turned and, with --store, quantised), attend -- from a CUDA
graph, and at the end the cached rows come back dense.

    python examples/decode_cache.py [--store e4m3|int8] [--steps 64]
        [--prefix 2000 | --pages 16 | --budget 512]

--prefix: all sequences begin with the same tokens, held and read once for all
of them.  --pages: a step attends over that many pages of each key head, those
whose bounds promise the largest scores.  --budget: steps add up the weight
that each token draws, and every eighth step the lightest beyond that many go,
the last 16 apart.

The model is one layer of random projections; what it shows is the order of
the calls and who owns which buffer.
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import layout_driven_movement_gb300 as lm


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--store", choices=("e4m3", "int8"))
    ap.add_argument("--steps", type=int, default=64)
    form = ap.add_mutually_exclusive_group()
    form.add_argument("--prefix", type=int, default=0)
    form.add_argument("--pages", type=int, default=0)
    form.add_argument("--budget", type=int, default=0)
    args = ap.parse_args(argv)
    if args.budget and args.budget < 16:
        ap.error("--budget: 16 at least")
    torch.manual_seed(0)
    dev, dtype = "cuda", torch.bfloat16
    heads, group, dim, page = 8, 4, 128, 16
    prompts = [700, 33, 1, 4000]
    seqs, heads_q = len(prompts), heads * group

    # the cache: a page is a layout of (tokens, heads, dim); every sequence
    # gets the pages that it will need out of one pool
    plan = lm.KVPlan(lm.Layout.parse(f"({page},{heads},{dim}):"
                                     f"({heads * dim},{dim},1)"),
                     dtype, args.store)
    most = -(-(max(prompts) + args.steps) // page)
    ahead = -(-args.prefix // page)         # pages of the shared prefix
    pool = ahead + seqs * most
    held = torch.zeros(2, pool, plan.page_stride, device=dev,
                       dtype=torch.uint8 if args.store else dtype)
    scales = torch.ones(2, pool, heads, page, device=dev) if args.store \
        else (None, None)
    cache = lm.KVCache(plan, held[0], held[1], scales[0], scales[1])
    pages = torch.randperm(pool, device=dev).int()
    shared = pages[:ahead].view(1, ahead)
    pages = pages[ahead:].view(seqs, most)

    rope = lm.RopePlan(dim, scaling="yarn", factor=4.0,
                       original_positions=2048)
    table = torch.empty(args.prefix + max(prompts) + args.steps, dim,
                        device=dev)
    lm.rope_table(rope, table)

    def slots_of(seq, pos):
        return pages[seq, pos // page].long() * page + pos % page

    # the prompts, all tokens in one ragged call
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    seq = torch.repeat_interleave(torch.arange(seqs, device=dev), lens.long())
    starts = torch.cat([lens.new_zeros(1), lens.cumsum(0).int()])
    pos = torch.arange(len(seq), device=dev) - starts[seq].long()
    kv = torch.randn(len(seq), 2 * heads, dim, device=dev).to(dtype)
    lm.kv_write(cache, kv[:, :heads], kv[:, heads:], slots_of(seq, pos),
                rope=rope, positions=pos + args.prefix, table=table)
    if args.prefix:
        kv = torch.randn(args.prefix, 2 * heads, dim, device=dev).to(dtype)
        pos = torch.arange(args.prefix, device=dev)
        lm.kv_write(cache, kv[:, :heads], kv[:, heads:],
                    shared[0, pos // page].long() * page + pos % page,
                    rope=rope, positions=pos, table=table)
        shared_lens = torch.tensor([args.prefix], dtype=torch.int32,
                                   device=dev)
        groups = torch.tensor([0, seqs], dtype=torch.int32, device=dev)

    # one step, captured: every buffer stays where it is
    width = heads_q * dim
    mix = (torch.randn(width, width + 2 * heads * dim, device=dev) /
           width ** 0.5).to(dtype)
    x = torch.randn(seqs, width, device=dev).to(dtype)
    q = torch.empty(seqs, heads_q, dim, dtype=dtype, device=dev)
    out = torch.empty_like(q)
    lse = torch.empty(seqs, heads_q, device=dev)
    step_pos = lens.long() + args.prefix
    rows = torch.arange(seqs, device=dev)

    def space(size, *size_args, **sizes):
        return torch.zeros(size(plan, *size_args, **sizes), dtype=torch.uint8,
                           device=dev)
    if args.prefix:
        workspace = space(lm.kv_attend_shared_workspace, seqs, heads_q)
    else:
        workspace = space(lm.kv_attend_workspace, seqs, heads_q,
                          max_pages=most)
    if args.pages:
        # the bounds of every page that holds something
        bounds = torch.zeros(pool, heads, 2, dim, dtype=torch.int8, device=dev)
        by = torch.ones(pool, heads, device=dev)
        counts = (lens[:, None] - torch.arange(most, device=dev).int() *
                  page).clamp(0, page)
        lm.kv_bound(cache, pages.flatten(), counts.flatten(), bounds, by)
        chosen = torch.empty(seqs, heads, args.pages, dtype=torch.int32,
                             device=dev)
        chosen_lens = torch.empty_like(lens)
        scores = space(lm.kv_select_workspace, seqs, most)
    if args.budget:
        weights = torch.zeros(pool, heads, page, device=dev)
        nothing = torch.zeros((), device=dev)
        kept = space(lm.kv_evict_workspace, seqs, args.budget)

    def step():
        fused = (x @ mix).view(seqs, heads_q + 2 * heads, dim)
        lm.rope(rope, fused[:, :heads_q], step_pos, table, q)
        slots = slots_of(rows, lens.long())
        lm.kv_write(cache, fused[:, heads_q:heads_q + heads],
                    fused[:, heads_q + heads:], slots,
                    rope=rope, positions=step_pos, table=table)
        lens.add_(1)
        step_pos.add_(1)
        if args.prefix:
            lm.kv_attend_shared(cache, q, shared, shared_lens, groups, pages,
                                lens, out, workspace, lse=lse)
        elif args.pages:
            lm.kv_bound(cache, (slots // page).int(),
                        (slots % page + 1).int(), bounds, by)
            lm.kv_select(cache, q, bounds, by, pages, lens, chosen,
                         chosen_lens, scores)
            lm.kv_attend(cache, q, chosen, chosen_lens, out, workspace,
                         lse=lse)
        elif args.budget:
            # (a token that has gone may have left its weight in the slot)
            weights[slots // page, :, slots % page] = nothing
            lm.kv_attend(cache, q, pages, lens, out, workspace, lse=lse,
                         weights=weights)
        else:
            lm.kv_attend(cache, q, pages, lens, out, workspace, lse=lse)
        x.copy_(torch.nn.functional.normalize(
            out.view(seqs, width).float(), dim=1) * width ** 0.5)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()                              # loads what a first call loads
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    torch.cuda.current_stream().wait_stream(stream)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for i in range(args.steps - 1):
        if args.budget and i % 8 == 0:
            lm.kv_evict(cache, weights, pages, lens, pages, lens, args.budget,
                        kept, recent=16)
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    us = a.elapsed_time(b) * 1000 / max(1, args.steps - 1)

    # what the cache holds, dense
    def dense(table, lens):
        starts = torch.cat([lens.new_zeros(1), lens.cumsum(0).int()])
        k = torch.empty(int(starts[-1]), heads, dim, dtype=dtype, device=dev)
        v = torch.empty_like(k)
        lm.kv_read(cache, table, lens, starts, k, v)
        parts = lens.tolist()
        return list(zip(k.float().split(parts), v.float().split(parts)))

    if args.pages:                          # each head has pages of its own
        by_head = [dense(chosen[:, h].contiguous(), chosen_lens)
                   for h in range(heads)]
        held = [tuple(torch.stack([by_head[h][i][kv][:, h]
                                   for h in range(heads)], 1)
                      for kv in (0, 1)) for i in range(seqs)]
    else:
        held = dense(pages, lens)
    if args.prefix:
        first = dense(shared, shared_lens)[0]
        held = [tuple(torch.cat([first[kv], own[kv]]) for kv in (0, 1))
                for own in held]
    status = lm.device_status()
    assert status == 0, lm.STATUS[status]
    # the last step again, plainly, over the rows that came back
    worst = 0.0
    for i in range(seqs):
        ki, vi = (t.repeat_interleave(group, 1) for t in held[i])
        p = torch.softmax(torch.einsum("hd,nhd->hn", q[i].float(), ki) *
                          dim ** -0.5, -1)
        want = torch.einsum("hn,nhd->hd", p, vi)
        worst = max(worst, ((out[i].float() - want).norm() /
                            want.norm()).item())
    print(f"{seqs} sequences of {lens.tolist()} tokens, store "
          f"{args.store or 'same'}: {us:.1f} us a step; last outputs within "
          f"{worst:.1e} of plain attention over the rows read back")
    return worst


if __name__ == "__main__":
    main()
