"""The serving example's global model: a prompt of chunks then single chunks give the rows that
the longer prompt gives, behind the encoder and the chunker, and go back to bytes."""
import numpy as np
import pytest

from tests.helpers import row_rel_err, to_np
from tests.test_gpu_mixer_example import _example

pytestmark = pytest.mark.gpu


def test_chunks_then_steps_equal_the_longer_prompt():
    import torch
    m = _example()
    model = m.GlobalModel(2, 9, 200)
    gen = torch.Generator(device="cuda").manual_seed(5)
    lengths, tail = [150, 3, 64, 65], 2
    off = np.cumsum([0] + lengths)
    rows = torch.randn(int(off[-1]), m.D, device="cuda", generator=gen).to(torch.bfloat16)
    slots = torch.tensor([7, 0, 3, 8], device="cuda", dtype=torch.int32)
    want = to_np(model.prompt(rows, torch.from_numpy(off).cuda(), slots))
    head = np.concatenate([np.arange(off[s], off[s + 1] - tail) for s in range(4)])
    model.prompt(rows[torch.from_numpy(head).cuda()], torch.from_numpy(np.cumsum([0] + [n - tail for n in lengths])).cuda(), slots)
    for i in range(tail):
        at = off[1:] - tail + i
        got = to_np(model.step(rows[torch.from_numpy(at).cuda()], slots))
        # keys and values of the steps are in 8 bits: off by up to half a step of 1/127 of a row's largest
        # value, some 3.3 times its typical one, evenly: 3.3 / 127 / sqrt(12) = 0.75 % a value; that
        # and the norms' 8 bits (as much again) over two blocks
        assert row_rel_err(got, want[at]) < 0.04
    assert torch.equal(model.lengths[slots.long()].cpu(), torch.tensor(lengths, dtype=torch.int32))
    assert int(model.lengths.sum()) == sum(lengths)


def test_bytes_to_chunks_to_bytes():
    import torch
    import byte_level_lm_amd as B
    m = _example()
    data = m.streams_of_bytes(np.random.default_rng(4), 3, 300)
    packed = torch.from_numpy(np.concatenate(data).astype(np.int64)).cuda()
    off = torch.from_numpy(np.cumsum([0] + [len(d) for d in data])).cuda()
    slots = torch.arange(3, device="cuda", dtype=torch.int32)
    enc, model = m.Encoder(1, 3), m.GlobalModel(1, 3, 301)
    idx, chunk_offsets, rows, P, status = enc.chunks(enc.prompt(packed, off, slots), off)
    n = int(chunk_offsets[-1])
    y = model.prompt(rows[:n], chunk_offsets, slots)
    out = B.dechunk_ema(y, P, idx, chunk_offsets, off, len(packed))
    assert int(status) == 0 and out.shape == (len(packed), m.D) and torch.isfinite(out.float()).all()
    # a byte's row is its chunk's average: the rows of the first chunk's bytes are the same
    first = int(idx[1]) if n > 1 else len(packed)
    assert torch.equal(out[:first], out[:1].expand(first, -1))
