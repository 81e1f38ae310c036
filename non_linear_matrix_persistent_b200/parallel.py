"""Multi-GPU plumbing over torch.distributed (one process per GPU).

Every (b, h) pair of the recurrence is independent, so ranks can shard it
two ways with no exchange inside the forward or backward kernels:
* the batch (data parallel): the one exchange is the gradient of the shared
  per-head W, a sum over the global batch, so each rank's dW (already summed
  over its own batch rows) is all-reduced (allreduce_dW; a norm's dweight and
  dbias, and the df of gates that are one constant per head, are such sums too);
* the heads, a whole number of k / q head groups per rank (the topology-aware
  tensor-parallel strategy of the pages, gist.science technical summary §2.2):
  a rank holds its groups' k and q and their heads' v, f, W and state, so
  nothing at all is exchanged (head_shard).
Linear attention and the readout norm are sharded the same two ways.
"""
from __future__ import annotations

import datetime
import os

import torch


def init(backend: str, timeout_s: int = 120):
    """Initialises the default process group from the torchrun environment
    (RANK, WORLD_SIZE, MASTER_ADDR, MASTER_PORT); returns (rank, world)."""
    import torch.distributed as dist
    if not dist.is_initialized():
        dist.init_process_group(backend, timeout=datetime.timedelta(seconds=timeout_s))
    return dist.get_rank(), dist.get_world_size()


def world_from_env():
    return int(os.environ.get("RANK", "0")), int(os.environ.get("WORLD_SIZE", "1"))


def allreduce_dW(dW: torch.Tensor) -> torch.Tensor:
    """In-place sum of the per-rank dW over all ranks (no-op on one rank)."""
    import torch.distributed as dist
    if dist.is_available() and dist.is_initialized() and dist.get_world_size() > 1:
        dist.all_reduce(dW, op=dist.ReduceOp.SUM)
    return dW


def max_over_ranks(x: float, device=None) -> float:
    import torch.distributed as dist
    if not (dist.is_available() and dist.is_initialized()) or dist.get_world_size() == 1:
        return x
    t = torch.tensor([x], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


# Where a problem's tensors hold their heads: the second dimension, except
_HEADS_FIRST = ("W", "dW", "weight", "bias", "dweight", "dbias")    # one row (or matrix) for each head
_HEADS_THIRD = ("n", "dn")                                          # a norm's token-first rows and their gradient
_PER_GROUP = ("k", "q", "dk", "dq")                                 # G groups, not H heads


def head_shard(x: dict, rank: int, world: int) -> dict:
    """The part of a problem that rank `rank` of `world` holds when heads are
    sharded: head groups [r·G/N, (r+1)·G/N) of k, q (and dk, dq) and the heads
    of those groups of every per-head tensor: v, f, W, H0, HT, dY, y, dv, df,
    dW, dH0, ckpt, linear attention's S0, ST, dST, dS0 (f and df may be [H]), a
    readout norm's x, dx, mean, rstd, its weight, bias, dweight, dbias ([H, N])
    and, token-first, its rows n and their gradient dn.  G is k's head count
    (= H when k and q are per head) and must be a multiple of world.  Returns
    contiguous slices; None stays None."""
    G, H = x["k"].shape[1], x["v"].shape[1]
    if G % world or H % G:
        raise ValueError("%d k/q head groups of %d heads cannot be split over %d ranks" % (G, H, world))
    out = {}
    for n, t in x.items():
        if t is None:
            out[n] = None
            continue
        heads = G if n in _PER_GROUP else H
        dim = 0 if n in _HEADS_FIRST or (n in ("f", "df") and t.dim() == 1) else 2 if n in _HEADS_THIRD else 1
        if n in _HEADS_FIRST and t.dim() < 2 or t.dim() <= dim or t.shape[dim] != heads:
            raise ValueError("%s has shape %s: %d heads are expected in dimension %d" % (n, tuple(t.shape), heads, dim))
        out[n] = t.narrow(dim, rank * heads // world, heads // world).contiguous()
    return out
