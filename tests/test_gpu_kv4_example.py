"""The decoder example, all operators together: forks, chunks, windows and compaction change nothing that they should
not, and a layer's attention is the plain one over the cache's values."""
import importlib.util
import os

import pytest
import torch

import quantized_matmul_quantize_amd as qmm

pytestmark = pytest.mark.gpu
spec = importlib.util.spec_from_file_location(
    "kv4_decode", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kv4_decode.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def decoder(**kw):
    return example.Decoder(**{**dict(layers=2, hidden=512, q_heads=8, kv_heads=2, head_dim=64, pages=64, page=16, group=32,
                                     rows=512), **kw})


def rows(n, seed):
    return torch.randn((n, 512), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_forks_and_compaction_change_nothing(window, sinks):
    """The same prompt and inputs, once straight on and once forked, moved and with a branch beside it."""
    a, b = decoder(window=window, sinks=sinks), decoder(window=window, sinks=sinks)
    sa, gone, sb = a.pages.add(), b.pages.add(), b.pages.add()
    b.step([gone], rows(40, 9), [40])
    prompt = rows(45, 1)
    assert torch.equal(a.step([sa], prompt, [45]), b.step([sb], prompt, [45]))
    branch = b.pages.fork(sb)
    for step in range(20):
        x, other = rows(1, 10 + step), rows(1, 50 + step)
        want = a.step([sa], x, [1])
        got = b.step([sb, branch], torch.cat([x, other]), [1, 1])
        # (one and two tokens take different kernels for the projections)
        tol = 2 ** -8 * (want.float().abs().max() + 1)
        assert (want.float() - got[:1].float()).abs().max() <= 8 * tol
        if step == 5:
            b.pages.free(gone)
            src, dst = b.pages.compact()
            assert len(src) > 0
            before = [b.cache[:, int(p)].clone() for p in src]
            b.copy(src, dst)
            assert all(torch.equal(b.cache[:, int(p)], x) for p, x in zip(dst, before))
    assert b.pages.length(sb) == b.pages.length(branch) == 65


@pytest.mark.parametrize("chunks", [[90], [64, 26], [33, 1, 56]])
def test_attention_of_a_layer_is_the_plain_one(chunks):
    """Against float64 softmax attention over kv4_read's values, for a prompt read in chunks."""
    m = decoder(layers=1)
    s = m.pages.add()
    seen = []
    real = qmm.kv4_attention
    try:
        def keep(q, *args, **kw):
            out = real(q, *args, **kw)
            seen.append((q, out))
            return out
        qmm.kv4_attention = keep
        x = rows(sum(chunks), 2)
        at = 0
        for n in chunks:
            m.step([s], x[at:at + n], [n])
            at += n
    finally:
        qmm.kv4_attention = real
    table, context = m.pages.table([s])
    j = torch.arange(int(context[0]))
    slots = table[0].long()[j // 16] * 16 + j % 16
    k, v = (y.double().cpu().repeat_interleave(4, 1) for y in qmm.kv4_read(m.cache[0], slots.cuda(), 64, dtype=torch.float32))
    q, out = (torch.cat([pair[i] for pair in seen]).double().cpu() for i in (0, 1))
    for h in range(8):
        score = q[:, h] @ k[:, h].T / 8
        score = score.masked_fill(j[None, :] > j[:, None], float("-inf"))
        want = torch.softmax(score, -1) @ v[:, h]
        # bf16's half step of the result, and as much of the sum of magnitudes
        bound = 2 ** -9 * want.abs() + 2 ** -8 * (torch.softmax(score, -1) @ v[:, h].abs())
        assert ((out[:, h] - want).abs() <= bound).all()


def test_the_command(capsys):
    x = example.main("--layers 2 --hidden 512 --q-heads 8 --kv-heads 2 --head-dim 64 --page 16 --sequences 3 --branches 2 "
                     "--prompt 70 --chunk 32 --steps 5 --window 40 --sinks 4".split())
    assert x.shape == (6, 512) and bool(torch.isfinite(x).all())
    text = capsys.readouterr().out
    assert "prompts: 3 x 70 tokens" in text and "6 branches" in text
