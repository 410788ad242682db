"""The serving example's path: prompts then single bytes give the rows that the
longer prompts give, its rows feed the chunker, and the command runs."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest

from tests.helpers import row_rel_err, to_np

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixer_serving.py")


def _example():
    spec = importlib.util.spec_from_file_location("mixer_serving", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_prompt_then_steps_equal_the_longer_prompt():
    import torch
    m = _example()
    data = m.streams_of_bytes(np.random.default_rng(3), 5, 200)
    tail = 3
    enc = m.Encoder(2, 9)
    slots = torch.tensor([7, 0, 3, 8, 4], device="cuda", dtype=torch.int32)

    def packed(parts):
        return (torch.from_numpy(np.concatenate(parts).astype(np.int64)).cuda(),
                torch.from_numpy(np.cumsum([0] + [len(p) for p in parts])).cuda())

    whole, off = packed(data)
    want = to_np(enc.prompt(whole, off, slots))
    ends = np.asarray(off.cpu())[1:]
    head, hoff = packed([d[:-tail] for d in data])
    enc.prompt(head, hoff, slots)
    for i in range(tail):
        got = to_np(enc.step(torch.tensor([int(d[len(d) - tail + i]) for d in data], device="cuda"), slots))
        # the two forms round o apart by 2^-9 a value; where that tips an 8-bit code, by a step of
        # 1/127 of the row's largest value, under 4 % of its typical one, on a part of the codes
        assert row_rel_err(got, want[ends - tail + i]) < 0.04
    # the rows feed the chunker: one boundary at every stream's start
    idx, chunk_offsets, rows, P, st = enc.chunks(enc.prompt(whole, off, slots), off)
    n = int(chunk_offsets[-1])
    assert int(st) == 0 and set(np.asarray(off.cpu())[:-1]) <= set(to_np(idx)[:n].tolist())


def test_the_command_runs():
    r = subprocess.run([sys.executable, PATH, "--streams", "4", "--longest", "128", "--steps", "2"],
                       capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "chunks in" in r.stdout and "us a byte" in r.stdout
