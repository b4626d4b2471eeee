"""Profile summaries name the sources that they were taken on, whatever their file is called."""
import os
import re

import pytest

PROFILES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles")


def _text(name):
    with open(os.path.join(PROFILES, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(PROFILES) if _text(n).startswith("# ncu summary")))
def test_ncu_summaries_name_their_sources(name):
    text = _text(name)
    assert re.search(r"(?m)^source_sha256: [0-9a-f]{16}$", text), name
    assert re.search(r"(?m)^ncu .*--clock-control none", text), name
