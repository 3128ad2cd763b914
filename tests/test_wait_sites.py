"""A device wait that runs out is reported by its site: every site of the
kernels has a number of its own and a name in the host's table."""
import glob
import os
import re

from windowed_attention_b200.build import CSRC


def _sources():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            yield os.path.basename(path), re.sub(r"//[^\n]*", "", f.read())


def test_every_site_has_a_number_and_a_name_of_its_own():
    at, names = {}, {}
    for name, text in _sources():
        for site, number in re.findall(r"\b(SITE_\w+)\s*=\s*(\d+)", text):
            assert number not in at, f"{number}: {name} {site} and {at[number]}"
            at[number] = f"{name} {site}"
        if name == "rib_api.cu":
            names = dict(re.findall(r'case (\d+): return "([^"]+)";', text))
        else:
            # no wait names its site by a bare number
            assert not re.search(r"mbar_wait\([^;]*,\s*\d{3}\)", text), name
    assert len(at) > 50
    missing = {n: s for n, s in at.items() if n not in names}
    assert not missing, missing
    assert len(set(names.values())) == len(names)
