"""Fresh outputs of a packed batch with bad offsets: what no sequence writes is zero, states too."""
import ctypes

import pytest
import torch

import metaplastic_linear_attention_gb300 as pal
from metaplastic_linear_attention_gb300 import ssm
from tests.test_ssm_gpu import BF, DEV, F32, _conv_inputs, _dev, _scan_inputs

pytestmark = pytest.mark.gpu
D, N, W = 136, 16, 4


def _used(*shapes):
    """Leaves the allocator with blocks of these shapes that hold NaN."""
    held = [torch.full(s, float("nan"), dtype=t, device=DEV) for s in shapes for t in (F32, BF) for _ in range(4)]
    torch.cuda.synchronize()
    del held


def _outputs(cu, rows, longest, dtype, seed=2):
    """Every operator's fresh outputs: (name, tensor, whether it has a row per token)."""
    n = len(cu) - 1
    i = _dev(_scan_inputs(seed, rows, n, D, 1, N, dtype))
    c = _dev(_conv_inputs(seed, rows, n, D, W, dtype))
    kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_seqlen=longest)
    dy = torch.ones(rows, D, dtype=dtype, device=DEV)
    shapes = ((rows, D), (rows, 1, N), (n, D, N), (n, W - 1, D))
    out = []
    _used(*shapes)
    y, st = pal.palimpsa_causal_conv(*c.values(), **kw)
    out += [("conv y", y, True), ("conv state_T", st, False)]
    _used(*shapes)
    g = pal.palimpsa_causal_conv_backward(*c.values(), dy, **kw)
    out += [("conv dx", g["dx"], True), ("conv dstate0", g["dstate0"], False)]
    _used(*shapes)
    y, h = pal.palimpsa_selective_scan(*i.values(), **kw)
    out += [("scan y", y, True), ("scan h_T", h, False)]
    ckpt = torch.zeros(pal.palimpsa_selective_scan_checkpoint_shape(n, rows, D, N, True), device=DEV)
    _used(*shapes)
    y, h, _ = pal.palimpsa_selective_scan_checkpointed(*i.values(), ckpt=ckpt, **kw)
    out += [("checkpointed y", y, True), ("checkpointed h_T", h, False)]
    _used(*shapes)
    g = pal.palimpsa_selective_scan_backward(*i.values(), ckpt, dy, **kw)
    out += [("scan " + k, g[k], True) for k in ("dx", "ddt", "dz", "dB", "dC")] + [("scan dh0", g["dh0"], False)]
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cu,longest", [
    (40, [0, 18, 19, 40, 44, 50], 12), (20, [0, 9, 5, 20], 20), (20, [-1, 4, 8, 12], 12), (0, [0, 3, 0], 0)])
def test_states_of_skipped_sequences_are_zero(dtype, rows, cu, longest):
    ok = torch.tensor([0 <= a <= b <= rows and b - a <= longest for a, b in zip(cu, cu[1:])])
    out = _outputs(cu, rows, longest, dtype)
    assert pal.palimpsa_get_device_status() == 5
    for name, t, per_token in out:
        assert torch.isfinite(t).all(), name
        if not per_token:
            assert not t[~ok].any() and t[ok].flatten(1).any(1).all(), name


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("where", [0, 300, 697])
def test_sequences_that_out_of_order_offsets_make_overlap_leave_nothing_unwritten(dtype, where):
    """Hundreds of sequences, and two that hold 600 and 900 of 1000 rows between them: where the batch's pieces are laid out
    close, the second does not fit. Its rows, and its state, are its own results or zeros."""
    cu = [0] * (where + 1) + [600, 100] + [1000] * (698 - where)
    for name, t, _ in _outputs(cu, 1000, 1000, dtype):
        assert torch.isfinite(t).all(), name
    assert pal.palimpsa_get_device_status() == 5


def test_whole_batches_keep_their_states():
    cu = [0, 5, 5, 40]
    for name, t, per_token in _outputs(cu, 40, 35, F32):
        assert torch.isfinite(t).all(), name
        if name.endswith(("state_T", "h_T")):            # the empty sequence's is the one it came with
            assert t.flatten(1).any(1).all(), name
    assert pal.palimpsa_get_device_status() == 0


@pytest.mark.parametrize("count", [1, 2, 300, 4096, 4097, 9001])
@pytest.mark.parametrize("back", [None, 0.0, 0.5, 1.0])
def test_zero_unwritten_by_itself(count, back):
    """Rows and entries as they are, but for those outside the sequences and of skipped ones; with an offset that steps
    back (the first, one in the middle, the last) all are zeroed."""
    g = torch.Generator().manual_seed(count)
    lens = torch.randint(0, 4, (count,), generator=g)
    lens[torch.randint(0, count, (3,), generator=g)] = 9                  # longer than max_seqlen
    cu = torch.cat([torch.tensor([2]), 2 + lens.cumsum(0)]).to(torch.int32)
    rows, longest = int(cu[-1]) + 3, 8
    if back is not None:
        at = int(back * (count - 1))
        cu[at + 1] = cu[at] - 1
    step = (cu[1:] < cu[:-1]).any()
    kept = torch.zeros(rows, dtype=torch.bool)
    fine = torch.zeros(count, dtype=torch.bool)
    for n, (a, b) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        if not step and b - a <= longest:
            kept[a:b] = True
            fine[n] = True
    toks = [torch.full((rows, w), 7.0, device=DEV) for w in (4, 20)]
    states = [torch.full((count, w), 7.0, device=DEV) for w in (8, 36)]
    arr = lambda ts: (ctypes.c_void_p * len(ts))(*(t.data_ptr() for t in ts))  # noqa: E731
    wid = lambda ts: (ctypes.c_longlong * len(ts))(*(t.shape[1] * 4 for t in ts))  # noqa: E731
    cud = cu.to(DEV)
    ssm._call("palimpsa_zero_unwritten", toks[0].get_device(), arr(toks), wid(toks), 2, arr(states), wid(states), 2,
              cud.data_ptr(), count, rows, longest)
    for t, keep in [(t, kept) for t in toks] + [(t, fine) for t in states]:
        assert torch.equal(t.cpu(), 7.0 * keep[:, None].expand(t.shape))
