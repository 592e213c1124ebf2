"""Rotary positions of several axes through ``UlyssesRankAttention`` on 2 and 4 real ranks (gloo), against the oracle's
rotation around the emulated ranks; forwards that are refused between forward and backward; the layer's status."""
import dataclasses
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import usp_workloads as W
from dist_launch import HERE, ROOT, _free_port
from dist_rope_worker import frequencies, rope_positions
from gpu_util import assert_close, half_ulp_bf16, need_gpu
from oracle import serving as OS

CASES = [(W.Workload("rope_p2", B=1, S=128, Hq=4, Hkv=2, D=64, P=2, doc_mode="explicit", doc_lens=(50, 78)), 2),
         (W.Workload("rope_replicated_p4", B=1, S=128, Hq=8, Hkv=2, D=64, P=4, doc_mode="explicit", doc_lens=(70, 58)), 3),
         (W.Workload("rope_rows_p2", B=2, S=64, Hq=4, Hkv=4, D=64, P=2, doc_mode="explicit", doc_lens=(30, 34)), 1)]


def _ranks(w, ops, n_axes, tmpdir):
    out, port = os.path.join(str(tmpdir), w.name), _free_port()
    procs = [subprocess.Popen([sys.executable, os.path.join(HERE, "dist_rope_worker.py"), "--ops", ops, "--workload",
                               json.dumps(dataclasses.asdict(w)), "--axes", str(n_axes), "--out", out], cwd=ROOT,
                              env=dict(os.environ, RANK=str(r), WORLD_SIZE=str(w.P), LOCAL_RANK=str(r),
                                       MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), OMP_NUM_THREADS="1"),
                              stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for r in range(w.P)]
    try:
        logs = [p.communicate(timeout=300)[0] for p in procs]
    finally:
        for p in procs:
            if p.poll() is None:
                p.kill()
    for p, log in zip(procs, logs):
        assert p.returncode == 0, log[-4000:]
    return [dict(np.load(f"{out}.rank{r}.npz")) for r in range(w.P)]


def _bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def _reference(w, n_axes, rounded=lambda x: x):
    host = {n: W.bf16_to_f64(x) for n, x in W.qkv_do_shards(w).items()}
    freqs, axes = frequencies(w.D // 2, n_axes)
    pos = rope_positions(w, n_axes).reshape(n_axes, -1)
    turn = lambda x, back=False: OS.rope(x.reshape(-1, *x.shape[-2:]), pos, freqs, axes, back=back)[0].reshape(x.shape)
    f = oracle.ulysses_fwd(rounded(turn(host["q"])), rounded(turn(host["k"])), host["v"], W.position_ids_shards(w), w.causal, w.window_left,
                           None, None)
    g = oracle.ulysses_bwd(f, host["do"], w.causal, w.window_left, None, None)
    return {"o": f["o_seq"], "dq": turn(g["dq_seq"], True), "dk": turn(g["dk_seq"], True), "dv": g["dv_seq"]}, g


@pytest.mark.parametrize("w,n_axes", CASES, ids=[w.name for w, _ in CASES])
def test_ranks_turn_their_chunks(w, n_axes, tmp_path):
    ref, _ = _reference(w, n_axes)
    for r, got in enumerate(_ranks(w, "oracle", n_axes, tmp_path)):
        assert got["refused"][0] == 5 and got["status"].tolist() == [0, 11]
        for name, want in ref.items():
            err = np.abs(got[name] - want[r]).max()
            assert err <= 1e-12 * max(1.0, np.abs(want).max()), (name, r, err)


@pytest.mark.gpu
@pytest.mark.parametrize("w,n_axes", CASES[:2], ids=[w.name for w, _ in CASES[:2]])
def test_gpu_ranks_turn_their_chunks(w, n_axes, tmp_path):
    need_gpu()
    from ulysses_sequence_long_gb300 import _build
    _build.build()
    # The layer's attention takes q and k turned and rounded, as the reference here does.  The parity bar of the attention
    # (max abs 2e-2, relative L2 5e-3) is that of dQ and dK before they are turned back: an element takes the errors of
    # its pair, (|cos| + |sin|) <= sqrt 2 of the largest, and is rounded once more, 2^-8 of it at most.
    ref, g = _reference(w, n_axes, _bf16)
    for r, got in enumerate(_ranks(w, "library", n_axes, tmp_path)):
        assert got["refused"][0] == 5 and got["status"].tolist() == [0, 11]
        for name, want in ref.items():
            slack = None
            if name in ("dk", "dv") and w.Hkv < w.P:   # each replica's part is bf16 before they are summed
                slack = oracle.relayout_bwd(half_ulp_bf16(g[name + "_head"]), w.P, w.Hkv)[r]
                if name == "dk":                       # and a turned element takes those of its pair
                    slack = np.concatenate([slack[..., :w.D // 2] + slack[..., w.D // 2:]] * 2, -1)
            bar = dict(max_abs=2e-2 * 2 ** 0.5, rel_l2=5e-3 + 2.0 ** -8) if name in ("dq", "dk") else {}
            assert_close(f"{w.name} {name} rank {r}", got[name], want[r], slack=slack, **bar)
