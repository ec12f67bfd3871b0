"""What the decode driver's text tells a user to pass is what it takes."""
import dataclasses
import re

import pytest

pytest.importorskip("torch")


def test_attention_is_asked_for_as_the_text_says():
    from ternary_weight_decode_b200 import decode
    said = re.findall(r"``attention=([^`]+)``", decode.__doc__)
    assert said == ["PagedAttention(...)"]
    assert hasattr(decode.PagedAttention, "build")
    field = {f.name: f for f in dataclasses.fields(decode.DecodeModel)}["attention"]
    assert "PagedAttention" in str(field.type)
    m = decode.DecodeModel(0, 3, mode="fused", attention=decode.PagedAttention(max_ctx=8))
    assert m.launches_per_step() == 3 * 4 + 1 + 3 * 3
