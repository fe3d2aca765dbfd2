"""The bindings' docstrings name their own arguments."""

import inspect
import re

import pytest

from gaussian_splatting_differentiable_ewa_amd import _lib as L

BOUND = [f for n, f in vars(L).items() if n.startswith("gs_") and inspect.isfunction(f) and f.__doc__]


def named_optional(doc):
    """The compound names in what stands before "may be None", back to the clause's start."""
    for clause in re.findall(r"([^;.(]*)may be None", " ".join(doc.split())):
        yield from re.findall(r"\b[a-z]+_[a-z0-9_]+\b", clause)


@pytest.mark.parametrize("f", BOUND, ids=lambda f: f.__name__)
def test_optional_arguments_exist(f):
    for name in named_optional(f.__doc__):
        assert name in inspect.signature(f).parameters, name
