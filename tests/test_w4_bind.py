"""lora_w4_bind looks at what it is given: types, shapes that belong together, and
where the tensors are.  On the CPU, so that nothing wrong reaches a kernel."""
import pytest

torch = pytest.importorskip("torch")
import segmented_gathered_rank_amd as sgr  # noqa: E402

H_IN, H_OUT, GROUP = 256, 96, 64


def _parts(**over):
    p = dict(codes=torch.zeros(H_OUT, H_IN // 2, dtype=torch.uint8),
             scale=torch.zeros(H_IN // GROUP, H_OUT, dtype=torch.bfloat16), group=GROUP)
    p.update(over)
    return p


ZERO = torch.zeros(H_IN // GROUP, H_OUT, dtype=torch.uint8)
TABLE = torch.zeros(16, dtype=torch.bfloat16)

REFUSED = [
    ("codes of another type", dict(codes=torch.zeros(H_OUT, H_IN // 2, dtype=torch.int32)), "codes"),
    ("fp32 scales", dict(scale=torch.zeros(H_IN // GROUP, H_OUT)), "scale"),
    ("fp16 scales", dict(scale=torch.zeros(H_IN // GROUP, H_OUT, dtype=torch.float16)), "scale"),
    ("fp32 zero points", dict(zero=ZERO.float()), "zero"),
    ("fp32 table", dict(table=TABLE.float()), "table"),
    ("a list for a tensor", dict(scale=[[1.0]]), "scale"),
    ("codes in one row", dict(codes=torch.zeros(H_OUT * H_IN // 2, dtype=torch.uint8)), "codes"),
    ("scales in one row", dict(scale=torch.zeros(H_OUT, dtype=torch.bfloat16)), "scale"),
    ("too few codes for the groups", dict(codes=torch.zeros(H_OUT, H_IN // 2 - 16, dtype=torch.uint8)), "codes"),
    ("scales of fewer columns than codes", dict(scale=torch.zeros(H_IN // GROUP, H_OUT - 4, dtype=torch.bfloat16)),
     "scale"),
    ("no groups", dict(scale=torch.zeros(0, H_OUT, dtype=torch.bfloat16)), "scale"),
    ("zero points of fewer groups", dict(zero=ZERO[:-1]), "zero"),
    ("zero points of fewer columns", dict(zero=torch.zeros(H_IN // GROUP, H_OUT + 4, dtype=torch.uint8)[:, :H_OUT - 4],
                                          scale=torch.zeros(H_IN // GROUP, H_OUT + 4, dtype=torch.bfloat16)), "zero"),
    ("zero points of another row stride", dict(zero=torch.zeros(H_IN // GROUP, H_OUT + 4, dtype=torch.uint8)), "stride"),
    ("a short table", dict(table=TABLE[:15]), "table"),
    ("a table in two rows", dict(table=TABLE.view(2, 8)), "table"),
    ("both zero points and a table", dict(zero=ZERO, table=TABLE), "zero"),
    ("a group of 16", dict(group=16), "group"),
    ("strided codes", dict(codes=torch.zeros(H_OUT, H_IN, dtype=torch.uint8)[:, ::2]), "dense"),
    ("strided scales", dict(scale=torch.zeros(H_OUT, H_IN // GROUP, dtype=torch.bfloat16).t()), "dense"),
    ("tensors of the host", dict(), "GPU"),
    ("zero points of the host", dict(zero=ZERO), "GPU"),
]


@pytest.mark.parametrize("over,word", [r[1:] for r in REFUSED], ids=[r[0] for r in REFUSED])
def test_refused(over, word):
    with pytest.raises(ValueError, match=word):
        sgr.lora_w4_bind(**_parts(**over))
