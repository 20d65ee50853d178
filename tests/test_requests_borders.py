"""Adapters, probabilities and verification where one path ends and the next begins: what needs no GPU."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import requests_oracle_np as orc


@pytest.mark.parametrize("u,taken", [(1.0, True), (2.0, True), (np.inf, True), (0.5, True), (np.nan, True), (-1.0, True)])
def test_oracle_holds_random_numbers_below_one(u, taken):
    """A token as likely in the target as in the draft is accepted whatever the number is: below 1 they all are."""
    p = np.float32([[0.25, 0.75], [0, 1]])
    tokens, accepted = orc.verify(p, p[:1], np.int32([0]), np.int32([0, 1]), np.float32([u]), np.float32([u]))
    assert accepted[0] == taken and list(tokens) == [0, 1]
