"""Two outputs of one memory, whose bytes would depend on which workgroup is last, are refused on
the host."""
import pytest

torch = pytest.importorskip("torch")
from test_paged_messages import SHAPE, at, read, refused, rotate


def test_queries_and_keys_into_one_output():
    refused(rotate(over=dict(Ko=at(2))), SHAPE, "same output")
    refused(rotate(over=dict(Q=at(2), K=at(2), Ko=at(2)), Hkv=2), SHAPE, "same output")     # in place of one tensor


def test_keys_and_values_into_one_output():
    refused(read(over=dict(Vo=at(4))), SHAPE, "same output")
