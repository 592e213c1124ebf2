"""One rank of the multi-process tests of rotary positions, run as a child process by tests/test_distributed_rope.py.

The rank turns its own chunk by its own positions (several axes), forward and backward, over a gloo group; between the two
it tries forwards that have to be refused.  ``--ops oracle``: local steps and rotation of the fp64 oracle on the CPU;
``--ops library``: the library's kernels on cuda:0 (exchanges go through the host, so no kernel waits for another rank)."""
import argparse
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for d in (ROOT, os.path.join(ROOT, "tests")):
    if d not in sys.path:
        sys.path.insert(0, d)

import numpy as np  # noqa: E402
import torch  # noqa: E402
import torch.distributed as dist  # noqa: E402

import usp_workloads as W  # noqa: E402
from dist_rank_worker import OracleOps  # noqa: E402
from oracle import serving as OS  # noqa: E402
from ulysses_sequence_long_gb300.distributed import RankShape, UlyssesRankAttention  # noqa: E402


def frequencies(pairs, n_axes):
    rng = np.random.default_rng(pairs)
    return (10000.0 ** -rng.uniform(0, 1, pairs)).astype(np.float32), rng.integers(0, n_axes, pairs).astype(np.int32)


def rope_positions(w, n_axes):
    """int32 [n_axes][P][B][S/P], others on every rank."""
    return np.random.default_rng(w.S).integers(-50, 3000, (n_axes, w.P, w.B, w.S // w.P)).astype(np.int32)


class OracleRope:
    """Rotary on float64 CPU tensors."""

    def __init__(self, freqs, axes, n_axes):
        self.freqs, self.axes, self.n_axes, self.status = freqs, axes, n_axes, 0

    def _turn(self, x, positions, back):
        pos = positions.numpy().reshape(self.n_axes, -1)
        y, _ = OS.rope(x.numpy().reshape(-1, *x.shape[-2:]), pos, self.freqs, self.axes, back=back)
        return torch.from_numpy(y.reshape(x.shape))

    def forward(self, q, k, positions, out=None, stream=None):
        return self._turn(q, positions, False), self._turn(k, positions, False)

    def backward(self, dq, dk, positions, out=None, stream=None):
        return self._turn(dq, positions, True), self._turn(dk, positions, True)

    def read_status(self):
        return self.status


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--ops", choices=["library", "oracle"], required=True)
    ap.add_argument("--workload", required=True)
    ap.add_argument("--axes", type=int, required=True)
    ap.add_argument("--out", required=True)
    args = ap.parse_args()
    rank, world = int(os.environ["RANK"]), int(os.environ["WORLD_SIZE"])
    wd = json.loads(args.workload)
    wd["doc_lens"] = tuple(wd["doc_lens"])
    w = W.Workload(**wd)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    shape = RankShape(w.B, w.S, w.Hq, w.Hkv, w.D, w.P, w.causal, w.window_left)
    t = W.qkv_do_shards(w)
    pos = torch.from_numpy(np.ascontiguousarray(W.position_ids_shards(w)[rank]))
    turn = torch.from_numpy(np.ascontiguousarray(rope_positions(w, args.axes)[:, rank]))
    freqs, axes = frequencies(w.D // 2, args.axes)
    if args.ops == "oracle":
        rope = OracleRope(freqs, axes, args.axes)
        ua = UlyssesRankAttention(shape, ops=OracleOps(shape), rope=rope)
        x = {n: torch.from_numpy(W.bf16_to_f64(t[n][rank])) for n in t}
    else:
        from ulysses_sequence_long_gb300.pipeline import Rotary
        torch.cuda.set_device(0)
        rope = Rotary(torch.from_numpy(freqs).cuda(), torch.from_numpy(axes).cuda(), args.axes)
        ua = UlyssesRankAttention(shape, device="cuda:0", rope=rope)
        x = {n: t[n][rank].contiguous().cuda() for n in t}
        pos, turn = pos.cuda(), turn.cuda()
    o = ua.forward(x["q"], x["k"], x["v"], pos, rope_positions=turn)
    # refused on every rank, before any exchange: what the backward reads stays
    zero = torch.zeros_like(pos)
    refused = 0
    for q, k, v, p, r in ((x["q"], x["k"], x["v"], zero, turn.reshape(-1)[:turn.numel() // 2].contiguous()),
                          (x["q"], x["k"], x["v"][:, :-1].contiguous(), zero, torch.zeros_like(turn)),
                          (x["q"], x["k"], x["v"].float(), zero, torch.zeros_like(turn)),
                          (x["q"][:, 1:].contiguous(), x["k"], x["v"], zero, torch.zeros_like(turn)),
                          (x["q"], x["k"], x["v"], zero[:, 1:].contiguous(), torch.zeros_like(turn))):
        try:
            ua.forward(q, k, v, p, rope_positions=r)
        except (TypeError, ValueError):
            refused += 1
    dq, dk, dv, _ = ua.backward(x["do"])
    good = ua.read_status()
    if args.ops == "oracle":
        rope.status = 11
    else:
        torch.cuda.synchronize()
        rope.status.fill_(11)
    f64 = lambda a: a.detach().double().cpu().numpy()
    np.savez(f"{args.out}.rank{rank}.npz", o=f64(o), dq=f64(dq), dk=f64(dk), dv=f64(dv),
             refused=np.array([refused]), status=np.array([good, ua.read_status()]))
    dist.barrier()
    dist.destroy_process_group()


if __name__ == "__main__":
    main()
